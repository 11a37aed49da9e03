// Muon: momentum, an update made orthogonal by Newton-Schulz products, and the
// weights' step, over a list of matrices.
//
//   m = mu m + g';  u = g' + mu m (Nesterov) or m;  X = u / (|u|_F + eps), turned over if it is tall (r <= k)
//   each iteration:  A = X X^T;  B = b A + c A A;  X = a X + B X
//   p -= rate wd p + rate update_rms sqrt(max(rows, columns)) X
//
// The products run on tcgen05 with fp16 operands and fp32 accumulators: the
// singular values lie in [0, 1.3], so that fp16's range is enough (X starts
// multiplied by a power of two near sqrt(r), where its entries are about 1 /
// sqrt(k) as they are at the end). Small singular values grow 3.4 times an
// iteration, and what rounding X leaves in their directions grows with them: the
// first kRests of the X's are kept with about five bits more (their rests), which
// the sum a X + B X takes beside the product. A is kept less a multiple of the
// identity (Poly). A and B are symmetric: only tiles that meet the lower triangle
// are computed, and stored on both sides.
//
// Matrices of one size lie one behind the other in the workspace (a group): one
// tensor map with the matrix as its third coordinate serves them, and cuts
// tiles off at a matrix's end. One launch of a product serves every group of
// the list, and starts while the one before it still writes what it reads: its
// loads are ordinary ones, which the wait orders (read-only loads are for memory
// that nobody writes while the kernel lives). Each output tile is one
// accumulator, K ascending: a matrix's result does not depend on its list.
// Matrices of up to 128 rows whose X fits shared memory take one kernel for the
// whole step instead (muon_small_kernel).
#include "rlk_device.cuh"
#include "rlk_internal.h"
#include "rlk_sm100.cuh"
#include "rlk_tmap.h"

#include <cuda_fp16.h>
#include <atomic>
#include <algorithm>
#include <map>
#include <math.h>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

RLK_DEFINE_STRICT_PROBE(probe_muon_tu)

namespace rlk {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ elementwise passes
constexpr int kItems = 40;          // matrices a launch of an elementwise pass takes (an argument of 6 KB)
constexpr int kPassThreads = 256;
constexpr int kMaxPartials = 256;   // partial sums of squares of a matrix (each CTA of the start adds them)
constexpr int kMinChunk = 8192;     // elements a partial sums, at least
constexpr int kSide = 64;           // the passes' tiles

// p -= decay p + rate X: fp64 and one rounding each, in one order, so that a rate on the device gives the bytes of the same
// number from the host. One thread a matrix computes them: fp64 is slow here.
struct Rates {
    double lr_scale, weight_decay, update_rms, root;  // root: of the longer side
    __device__ __forceinline__ void get(double lr, float& rate, float& decay) const {
        lr *= lr_scale;
        rate = (float)(lr * update_rms * root);
        decay = (float)(lr * weight_decay);
    }
};

struct Item {
    void* p;          // step: fp32, or bf16 with master; orthogonalize: bf16 out
    float* master;
    const void* g;    // step: gradient; orthogonalize: the matrix
    float* m;         // null: orthogonalize
    __half* x;        // the matrix's X [r, ld]
    uint8_t* rest;    // what rounding it leaves [r, ld_rest]
    double* part;     // its partial sums
    long long n, chunk;
    int rows, cols, ld, ld_rest, parts, block0;
    float start;      // X's power of two at the start
    float* rates;     // step: where the first pass leaves the last one's rate and decay
    Rates rate;
    bool g32;
};
struct PassArgs {
    Item item[kItems];
    int n;
    float mu, eps;
    bool nesterov;
    double lr;
    const float *grad_scale, *lr_dev;  // lr_dev: read instead of lr
};

__device__ __forceinline__ const Item& item_of(const PassArgs& a) {
    int i = 0;
    while (i + 1 < a.n && (int)blockIdx.x >= a.item[i + 1].block0) ++i;
    return a.item[i];
}
// Eight neighbouring values from i on, those from `live` on zeros; kVec: all there and 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ void load8(float (&v)[8], const void* g, bool fp32, long long i, int live) {
    if (kVec) {
        if (fp32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
            const float4 a = p[0], b = p[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(w[k]), v[2 * k + 1] = bf16_hi(w[k]);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = k >= live ? 0.0f
               : fp32    ? static_cast<const float*>(g)[i + k]
                         : __uint_as_float((uint32_t)static_cast<const uint16_t*>(g)[i + k] << 16);
}
template <bool kVec>
__device__ __forceinline__ void store8(float* p, long long i, const float (&v)[8], int live) {
    if (kVec) {
        float4* q = reinterpret_cast<float4*>(p + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < live) p[i + k] = v[k];
}
// The factor of the gradients; false: it is not finite and the tensors stay as they are.
__device__ __forceinline__ bool factor_of(const PassArgs& a, float& f) {
    f = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    return fabsf(f) < INFINITY;
}
// |u| from the sum of its squares, at least 2^-56: fp32 squares of magnitudes below 2^-75 are 0, and as many of them as a
// matrix has come to 2^-59. (A quotient by less would make X as large as it likes with a small eps.)
__device__ __forceinline__ float norm_of(double squares) {
    const float n = sqrtf((float)squares);
    return n < 0x1p-56f ? 0x1p-56f : n;  // (a NaN stays)
}
// The sum over the CTA's threads, in a fixed order.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[kPassThreads / 32];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kPassThreads / 32; ++i) v += s[i];
    return v;
}

// New momentum, and the partial sums of u's squares: a chunk of consecutive elements a CTA, eight neighbours a thread
// and turn, four turns in fp32 (32 squares), then fp64, which is slow here.
__global__ void __launch_bounds__(kPassThreads) muon_momentum_kernel(const __grid_constant__ PassArgs a) {
    const Item& it = item_of(a);
    float f;
    if (!factor_of(a, f)) return;
    const int chunk = blockIdx.x - it.block0;
    const long long lo = chunk * it.chunk, hi = min(lo + it.chunk, it.n);
    auto eight = [&](auto vec, long long i, int live, float& sq) {
        constexpr bool kVec = decltype(vec)::value;
        float u[8];
        load8<kVec>(u, it.g, it.g32, i, live);
        if (it.m != nullptr) {
            float m[8];
            load8<kVec>(m, it.m, true, i, live);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float g = u[k] * f;
                m[k] = fmaf(a.mu, m[k], g);
                u[k] = a.nesterov ? fmaf(a.mu, m[k], g) : m[k];
            }
            store8<kVec>(it.m, i, m, live);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sq = fmaf(u[k], u[k], sq);
    };
    double sum = 0.0;
    // (chunks start at multiples of 8 elements: 16-byte aligned)
    for (long long i0 = lo + 8 * threadIdx.x; i0 < hi; i0 += 4 * 8 * kPassThreads) {
        float sq = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const long long i = i0 + t * 8 * kPassThreads;
            if (i + 8 <= hi)
                eight(std::true_type{}, i, 8, sq);
            else if (i < hi)
                eight(std::false_type{}, i, (int)(hi - i), sq);
        }
        sum += (double)sq;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) it.part[chunk] = sum;
    if (threadIdx.x == 32 && chunk == 0 && it.m != nullptr)
        it.rate.get(a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr, it.rates[0], it.rates[1]);
}

// A 64 x 64 tile of a matrix by 256 threads: thread t has eight columns of the rows t / 8 and t / 8 + 32, neighbours
// where rows are 16-byte aligned (kVec), else every eighth from t % 8 on: a warp's accesses then meet 32 bytes of a
// row at a time (2 x 4530 x 1875 beside 2 x 2560 x 7680: the update 186 -> 127 us).
struct TileOf {
    int r0, c0;
    __device__ __forceinline__ TileOf(const Item& it) {
        const int tiles_c = (it.cols + kSide - 1) / kSide, t = blockIdx.x - it.block0;
        r0 = t / tiles_c * kSide;
        c0 = t % tiles_c * kSide;
    }
};
template <bool kVec>
__device__ __forceinline__ int column_of(int k) {
    return kVec ? 8 * (threadIdx.x & 7) + k : (threadIdx.x & 7) + 8 * k;
}
// The values at column_of(0 .. 7) of a row from i on, of which `live` exist (kVec: all eight or none).
template <bool kVec>
__device__ __forceinline__ void load_row(float (&v)[8], const void* g, bool fp32, long long i, int live) {
    if (kVec) {
#pragma unroll
        for (float& x : v) x = 0.0f;
        if (column_of<true>(0) < live) load8<true>(v, g, fp32, i + column_of<true>(0), 8);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int c = column_of<false>(k);
        v[k] = c >= live ? 0.0f
               : fp32    ? static_cast<const float*>(g)[i + c]
                         : __uint_as_float((uint32_t)static_cast<const uint16_t*>(g)[i + c] << 16);
    }
}
// Where column c (0 .. 63) of row r of a turned tile lies in shared memory: 16-byte chunks exchanged by the row's
// group of 8, so that threads of eight neighbouring row groups meet other banks.
__device__ __forceinline__ int turned(int r, int c) { return r * kSide + ((((c >> 3) ^ (r >> 3)) & 7) << 3) + (c & 7); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What rounding X to fp16 leaves, as an e4m3 code of it times a power of two: five bits of it or so.
//
// The iteration takes a small singular value s to a s = 3.4 s, and a perturbation of X between two such directions
// likewise; one that meets a direction whose value has grown is multiplied by that value's own growth alone, which ends
// near 1. Rounding X spreads 2^-12 of its norm over all directions, so where a few of them lead, the others drown: X off
// by 5e-3 of its norm with four leading by 10 times, 2e-2 with one by 100, 9e-2 with three alone, and it is the roundings
// of the first X's that grow. B X and A do not pass them on (B is 0 but for directions that have grown), a X does. So
// a X alone takes the rests: with a in the first two iterations, from the third on, where most values have grown, with
// the coefficient that X itself has beside B (Poly). What a direction of eigenvalue t of A needs is a + b t + c t^2: with
// few rows much alike a is too much, so small matrices take t as a quarter of the mean (4 to 15 rows: 6.6e-4 of X for
// independent entries where a leaves 8e-4 to 1e-3 and no rests 5.8e-4; four leading by 30 times 1.3e-3, 1.1e-3, 9e-3), none of it
// for 2 and 3 rows (where one leads by 10^4 a quarter leaves 2e-2), all of it for one, whose eigenvalue it is. Three rests leave 4e-4 to 1.4e-3 of X up to 100 times (two 2e-3,
// four no less), 3e-3 to 7e-3 beyond; few rows or entries, whose roundings do not average out, up to 1.3e-2.
constexpr int kRests = 3;
// X's entries are 1 at most (times its power of two at the start): rests of 2^-12 and less, 448 and less times this, and
// those of entries of 2^-14 and more keep their bits.
constexpr float kRestScale = 1048576.0f;
// Small matrices at the start: X's entries are below 2^12 and mostly below 2^9, rests below 2 and 1/4.
constexpr float kRestScaleStart = 192.0f;
__device__ __forceinline__ uint32_t rests2(uint64_t x, __half2 h, float scale) {  // of two x, the first one's in the low byte
    const float2 f = __half22float2(h);
    float lo, hi;
    f2_unpack(mul_f2(sub_f2(x, f2_pack(f.x, f.y)), f2_pack(scale, scale)), lo, hi);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t rests2(float x0, float x1, __half2 h, float scale) { return rests2(f2_pack(x0, x1), h, scale); }
__device__ __forceinline__ float2 rest_values(uint32_t codes) {  // of the two low bytes
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint2 rests8(const float (&v)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; k += 2) w[k >> 2] |= rests2(v[k], v[k + 1], __floats2half2_rn(v[k], v[k + 1]), scale) << 8 * (k & 3);
    return make_uint2(w[0], w[1]);
}

// X = u * start / (|u| + eps) in fp16 and its rest, turned over where the matrix is tall.
template <bool kVec>
__global__ void __launch_bounds__(kPassThreads, 6) muon_start_kernel(const __grid_constant__ PassArgs a) {
    __shared__ __align__(16) __half tile[kSide * kSide];
    __shared__ __align__(8) uint8_t rests[kSide * kSide];
    __shared__ float s_inv;
    const Item& it = item_of(a);
    float f;
    const bool ok = factor_of(a, f);
    const TileOf at(it);
    const bool tall = it.rows > it.cols;
    float u[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = at.r0 + (threadIdx.x >> 3) + 32 * k, live = !ok || r >= it.rows ? 0 : min(it.cols - at.c0, kSide);
        const long long i = (long long)r * it.cols + at.c0;
        load_row<kVec>(u[k], it.g, it.g32, i, live);
        if (it.m != nullptr) {
            float m[8];
            load_row<kVec>(m, it.m, true, i, live);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[k][j] = a.nesterov ? fmaf(a.mu, m[j], u[k][j] * f) : m[j];
        }
    }
    // (one warp adds: fp64 is slow here; root and quotient in fp32, one rounding each)
    if (threadIdx.x < 32) {
        double sq = 0.0;
        for (int i = threadIdx.x; i < it.parts; i += 32) sq += it.part[i];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, k);
        if (threadIdx.x == 0) s_inv = it.start / (norm_of(sq) + a.eps);
    }
    __syncthreads();
    const float inv = s_inv, rest_scale = kRestScale / it.start;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int rr = (threadIdx.x >> 3) + 32 * k, r = at.r0 + rr;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[k][j] *= inv;
        if (kVec && !tall) {
            const int c = at.c0 + column_of<true>(0);
            if (r < it.rows && c < it.cols) {
                *reinterpret_cast<uint4*>(it.x + (long long)r * it.ld + c) = pack8(u[k]);
                *reinterpret_cast<uint2*>(it.rest + (long long)r * it.ld_rest + c) = rests8(u[k], rest_scale);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column_of<kVec>(j), to = tall ? turned(c, rr) : turned(rr, c);
            const __half h = __float2half_rn(u[k][j]);
            tile[to] = h;
            rests[to] = (uint8_t)rests2(u[k][j], 0.0f, __halves2half2(h, __float2half_rn(0.0f)), rest_scale);
        }
    }
    if (kVec && !tall) return;
    __syncthreads();
    const int rows = tall ? it.cols : it.rows, cols = tall ? it.rows : it.cols, r0 = tall ? at.c0 : at.r0, c0 = tall ? at.r0 : at.c0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // (a row's padding takes zeros)
        const int rr = (threadIdx.x >> 3) + 32 * k, r = r0 + rr, cc = 8 * (threadIdx.x & 7), col = c0 + cc;
        if (r < rows && col < cols) {
            *reinterpret_cast<uint4*>(it.x + (long long)r * it.ld + col) = *reinterpret_cast<const uint4*>(tile + turned(rr, cc));
            *reinterpret_cast<uint2*>(it.rest + (long long)r * it.ld_rest + col) = *reinterpret_cast<const uint2*>(rests + turned(rr, cc));
        }
    }
}

// p -= decay p + rate X, or p = X (orthogonalize).
template <bool kVec>
__global__ void __launch_bounds__(kPassThreads, 5) muon_update_kernel(const __grid_constant__ PassArgs a) {
    __shared__ __align__(16) __half tile[kSide * kSide];
    const Item& it = item_of(a);
    float f;
    if (!factor_of(a, f)) return;
    const TileOf at(it);
    const bool tall = it.rows > it.cols;
    float* const p = it.master != nullptr ? it.master : static_cast<float*>(it.p);
    // everything that is read, before anything is written
    uint4 x[2];
    float q[2][8];
    const int rows = tall ? it.cols : it.rows, cols = tall ? it.rows : it.cols, r0 = tall ? at.c0 : at.r0, c0 = tall ? at.r0 : at.c0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int rr = (threadIdx.x >> 3) + 32 * k, cc = 8 * (threadIdx.x & 7);
        x[k] = make_uint4(0, 0, 0, 0);
        if (r0 + rr < rows && c0 + cc < cols) x[k] = *reinterpret_cast<const uint4*>(it.x + (long long)(r0 + rr) * it.ld + c0 + cc);
    }
    if (it.m != nullptr) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = at.r0 + (threadIdx.x >> 3) + 32 * k;
            load_row<kVec>(q[k], p, true, (long long)r * it.cols + at.c0, r >= it.rows ? 0 : min(it.cols - at.c0, kSide));
        }
    }
    if (tall || !kVec) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(tile + turned((threadIdx.x >> 3) + 32 * k, 8 * (threadIdx.x & 7))) = x[k];
        __syncthreads();
    }
    const float rate = it.m != nullptr ? it.rates[0] : 0.0f, decay = it.m != nullptr ? it.rates[1] : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int rr = (threadIdx.x >> 3) + 32 * k, r = at.r0 + rr, live = r >= it.rows ? 0 : min(it.cols - at.c0, kSide);
        const long long i = (long long)r * it.cols + at.c0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column_of<kVec>(j);
            const float y = kVec && !tall ? __half2float(reinterpret_cast<const __half*>(&x[k])[j])
                                          : __half2float(tile[tall ? turned(c, rr) : turned(rr, c)]);
            v[j] = it.m != nullptr ? q[k][j] - fmaf(decay, q[k][j], rate * y) : y;
        }
        const bool both = it.m == nullptr || it.master != nullptr;
        uint16_t* const b = static_cast<uint16_t*>(it.p) + i;
        if (kVec) {
            if (column_of<true>(0) >= live) continue;
            if (it.m != nullptr) store8<true>(p, i + column_of<true>(0), v, 8);
            if (both)
                *reinterpret_cast<uint4*>(b + column_of<true>(0)) =
                    make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = column_of<false>(j);
                if (c >= live) continue;
                if (it.m != nullptr) p[i + c] = v[j];
                if (both) b[c] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
            }
        }
    }
}

// ------------------------------------------------------------------ products
enum Mode { kGram = 0, kPoly = 1, kApply = 2 };
constexpr int kGroups = 8;  // sizes a launch takes
// A cluster of two CTAs computes a tile of 256 rows (128 each) x 256 columns; each holds its rows' operand and half of
// the columns': the pair's products read half as much shared memory, and TMA brings 32 KB instead of 48 a k-step and
// CTA (one CTA a tile was bound by that: X X^T of four projections 136 -> 113 us, B X 206 -> 174, 1.5 PFLOP/s).
constexpr int kBM = 128, kBN = 256, kBK = 64, kStages = 6;
constexpr int kOutBytes = 32 * 32 * 2;  // an epilogue warp's buffer: 32 rows of 32 columns
constexpr int kThreads = 384;
constexpr int kABytes = kBM * kBK * 2, kStageBytes = kABytes + kBN / 2 * kBK * 2;
constexpr int kSmemBytes = kStages * kStageBytes + 8 * kOutBytes + 1024;
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpEpilogue = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ int g_status_muon;

struct Group {
    CUtensorMap map_m;   // the operand of the 128 rows: [z][rows][K], box 64 x 128 x 1
    CUtensorMap map_n;   // the operand of the kBN columns: gram, poly the same, box 64 x 128; apply X, box 64 x 64 (MN-major)
    CUtensorMap map_out; // out, box 32 x 32 x 1
    const __half* add;   // gram: the identity (not read); poly: D; apply: X: added times `add_by`
    __half* out;
    uint8_t* rest;       // apply: X's rests, or null; the new X's are written in their place (rest_out)
    bool rest_out;
    long long add_step, out_step, rest_step;  // from matrix to matrix
    int rows, cols;      // of the output (gram, poly: r x r)
    int ld_add, ld_out, ld_rest, count, steps, per, tile0;  // matrices; k-steps; tiles of one matrix; first tile
    float by, add_by, rest_by;  // out = by * product + add_by * add + rest_by * rest (as its code has it)
};
struct GemmArgs {
    Group g[kGroups];
    int n, tiles;
};

struct TileAt {
    int g, z, m0, n0;
};
// Tile t of a launch: its first row (of both CTAs) and column.
template <int kMode>
__device__ __forceinline__ TileAt tile_at(const GemmArgs& a, int t) {
    TileAt r;
    r.g = 0;
    while (r.g + 1 < a.n && t >= a.g[r.g + 1].tile0) ++r.g;
    const Group& g = a.g[r.g];
    int l = t - g.tile0;
    r.z = l / g.per;
    l -= r.z * g.per;
    if (kMode == kApply) {
        const int tn = (g.cols + kBN - 1) / kBN;
        r.m0 = l / tn * (2 * kBM);
        r.n0 = l % tn * kBN;
    } else {
        // i (i + 1) / 2 tiles before block row i
        int i = (int)((sqrtf(8.0f * l + 1.0f) - 1.0f) * 0.5f);
        while (i * (i + 1) / 2 > l) --i;
        while ((i + 1) * (i + 2) / 2 <= l) ++i;
        r.m0 = i * (2 * kBM);
        r.n0 = (l - i * (i + 1) / 2) * kBN;
    }
    return r;
}

__device__ __forceinline__ void fail(volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(&g_status_muon, 1);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitLimitNs));
}
// One iteration's polynomial in D = A - shift I, an identity for any shift:
//   a X + (b A + c A A) X = (a + b shift + c shift^2) X + ((b + 2 c shift) D + c D D) X
// A's diagonal, which holds most of it, is the squared norms of X's rows. With about their mean taken off it, little is
// rounded to fp16: near 1, where A's roundings were multiplied by b = -4.8 and B's were 2^-11 of 2.7, the two
// coefficients are 0.7 (X off by 4e-4 to 8e-4 of its norm, 1.0e-3 to 2.1e-3 without). Small matrices take the mean
// itself, X's squares summed. The larger ones, where it would take a sum over many CTAs, take kSpread / r and what the
// polynomial makes of it, 1 at most: a rule on r alone. 1 / r, the mean at the start, is too early where a few singular
// values lead (300 x 1000 and 700 x 1500 with four of them: 0.35 5.1e-4 and 5.9e-4, 1 5.2e-4 and 8.3e-4, 0.2 4.7e-4 and
// 5.1e-4, the mean the same; independent entries: 0.35 8.0e-4 and 6.6e-4, 1 and the mean 6.3e-4 and 6.1e-4, 0.2 9.4e-4
// and 7.5e-4).
constexpr float kSpread = 0.35f;
struct Poly {
    float a, b, c;
    __host__ __device__ float of_x(float shift) const { return fmaf(fmaf(c, shift, b), shift, a); }
    __host__ __device__ float of_d(float shift) const { return fmaf(2.0f * c, shift, b); }
};
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 columns from j on of row i (a warp: 32 rows from i - lane): out = by * v + add_by * add (gram: the identity), and
// on the other side of the diagonal; apply: + rest_by * rest, and the rest of what is stored.
template <int kMode>
__device__ __forceinline__ void store32(const Group& g, int z, float (&v)[32], int i, int j, uint32_t buffer) {
    const int lane = threadIdx.x & 31, i0 = i - lane;
    const bool live = i < g.rows;
    if (kMode != kGram) {
        const __half* add = g.add + z * g.add_step + (long long)i * g.ld_add + j;
        uint8_t* const rest = g.rest + z * g.rest_step + (long long)i * g.ld_rest + j;
        const bool rests = kMode == kApply && g.rest != nullptr;
        uint4 w[4], b[2];  // (everything that is read, before the rests are written)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[c] = make_uint4(0, 0, 0, 0);
            if (live && j + 8 * c < g.cols) w[c] = *reinterpret_cast<const uint4*>(add + 8 * c);
        }
        if (rests) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // (rows of rests have room up to a multiple of 16)
                b[c] = make_uint4(0, 0, 0, 0);
                if (live && j + 16 * c < g.cols) b[c] = *reinterpret_cast<const uint4*>(rest + 16 * c);
            }
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            const uint4& q = w[c >> 3];
            const uint32_t word = (c >> 1 & 3) == 0 ? q.x : (c >> 1 & 3) == 1 ? q.y : (c >> 1 & 3) == 2 ? q.z : q.w;
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&word));
            v[c] = fmaf(g.add_by, x.x, g.by * v[c]);
            v[c + 1] = fmaf(g.add_by, x.y, g.by * v[c + 1]);
        }
        if (rests) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                const uint4& q = b[c >> 4];
                const uint32_t word = (c >> 2 & 3) == 0 ? q.x : (c >> 2 & 3) == 1 ? q.y : (c >> 2 & 3) == 2 ? q.z : q.w;
                const float2 x = rest_values(word >> 8 * (c & 2));
                v[c] = fmaf(g.rest_by, x.x, v[c]);
                v[c + 1] = fmaf(g.rest_by, x.y, v[c + 1]);
            }
            if (g.rest_out) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t n[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 16; k += 2)
                        n[k >> 2] |= rests2(v[16 * c + k], v[16 * c + k + 1], __floats2half2_rn(v[16 * c + k], v[16 * c + k + 1]), kRestScale) << 8 * (k & 2);
                    if (live && j + 16 * c < g.cols) *reinterpret_cast<uint4*>(rest + 16 * c) = make_uint4(n[0], n[1], n[2], n[3]);
                }
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] *= g.by;
    }
    __half* out = g.out + z * g.out_step;
    __half* row = out + (long long)i * g.ld_out + j;
    if (kMode != kApply && j == i0) {  // on the diagonal: the lower triangle and its mirror image, value by value
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (live && c <= lane) {
                const __half h = __float2half_rn(kMode == kGram && c == lane ? v[c] + g.add_by : v[c]);
                row[c] = h;
                out[(long long)(j + c) * g.ld_out + i] = h;
            }
        return;
    }
    // the rows through the warp's buffer (64-byte rows, 16-byte chunk c at c ^ (row / 2) % 4) and TMA, which cuts off
    // what is past the matrix
    bulk_wait_read_all();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buffer + 64 * lane + 16 * (c ^ ((lane >> 1) & 3))),
                     "r"(pack_half(v[8 * c], v[8 * c + 1])), "r"(pack_half(v[8 * c + 2], v[8 * c + 3])),
                     "r"(pack_half(v[8 * c + 4], v[8 * c + 5])), "r"(pack_half(v[8 * c + 6], v[8 * c + 7]))
                     : "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && i0 < g.rows) {
        tma_store_3d(&g.map_out, buffer, j, i0, z);
        bulk_commit_group();
    }
    if (kMode == kApply) return;
    const bool odd = lane & 1;
    __half* col = out + (long long)(j + odd) * g.ld_out + (i & ~1);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        // (all columns here are below the warp's rows, so they exist; the pair may end in the row's padding)
        if ((i & ~1) < g.rows) *reinterpret_cast<uint32_t*>(col) = odd ? pack_half(got, v[c + 1]) : pack_half(v[c], got);
        col += 2 * g.ld_out;
    }
}

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) muon_gemm_kernel(const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = cluster_rank(), first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto stage_a = [&](int st) { return sbase + st * kStageBytes; };
    auto stage_b = [&](int st) { return sbase + st * kStageBytes + kABytes; };
    // (full and free: the first CTA's count for both)
    const uint32_t bar_full = smem_u32(&bars[0]), bar_empty = bar_full + 8 * kStages;
    const uint32_t bar_acc = bar_empty + 8 * kStages, bar_free = bar_acc + 16, bar_drain = bar_free + 16;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) mbar_init(bar_full + 8 * i, 1), mbar_init(bar_empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(bar_acc + 8 * i, 1), mbar_init(bar_free + 8 * i, 16);
        mbar_init(bar_drain, 1);
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    // (the kernel before this one still writes what the loads read; the one after may set itself up)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == kWarpTma) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n) {
                const TileAt at = tile_at<kMode>(a, t);
                const Group& g = a.g[at.g];
                const int m0 = at.m0 + kBM * rank, n0 = at.n0 + kBN / 2 * rank;
                for (int kk = 0; kk < g.steps; ++kk, ++it) {
                    const int st = it % kStages;
                    const uint32_t use = it / kStages, bar = bar_full + 8 * st;
                    if (use > 0 && !mbar_wait(bar_empty + 8 * st, (use - 1) & 1, &abort_flag, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_expect_tx(bar, 2 * kStageBytes);
                    tma_load_3d_pair(stage_a(st), &g.map_m, bar, kk * kBK, m0, at.z);
                    if (kMode == kApply) {
#pragma unroll
                        for (int q = 0; q < kBN / 128; ++q)
                            tma_load_3d_pair(stage_b(st) + q * 8192, &g.map_n, bar, n0 + 64 * q, kk * kBK, at.z);
                    } else {
                        tma_load_3d_pair(stage_b(st), &g.map_n, bar, kk * kBK, n0, at.z);
                    }
                }
            }
            if (!ok) fail(&abort_flag);
            // drain: what was issued here has landed (counted by the first CTA) or been consumed
            for (uint32_t u = it < kStages ? 0 : it - kStages; (rank == 0 || ok) && u < it; ++u)
                mbar_wait_drain((rank == 0 ? bar_full : bar_empty) + 8 * (u % kStages), (u / kStages) & 1, kWaitLimitNs);
        }
    } else if (warp == kWarpMma) {
        if (rank == 0) {
            // the whole warp runs the loop, one lane issues
            constexpr uint32_t idesc = idesc_f16(2 * kBM, kBN, kMode == kApply);
            const uint64_t a0 = sdesc_sw128(stage_a(0), 16, 1024);
            const uint64_t b0 = kMode == kApply ? sdesc_sw128(stage_b(0), 8192, 1024) : sdesc_sw128(stage_b(0), 16, 1024);
            constexpr int kStepB = (kMode == kApply ? 2048 : 32) >> 4;
            uint32_t st = 0, phase = 0, local = 0;
            bool ok = true;
            for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n, ++local) {
                const int buf = local & 1;
                const uint32_t use = local >> 1;
                if (use > 0 && !__all_sync(0xffffffffu, mbar_wait_cluster(bar_free + 8 * buf, (use - 1) & 1, &abort_flag, kWaitLimitNs))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + buf * kBN;
                const int steps = a.g[tile_at<kMode>(a, t).g].steps;
                for (int kk = 0; kk < steps; ++kk) {
                    if (!warp_wait(bar_full + 8 * st, phase, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = a0 + st * (kStageBytes >> 4), db = b0 + st * (kStageBytes >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j) mma_pair(acc, da + 2 * j, db + kStepB * j, idesc, (kk > 0 || j > 0) ? 1u : 0u);
                        mma_commit_pair(bar_empty + 8 * st);
                    }
                    if (++st == kStages) st = 0, phase ^= 1;
                }
                if (ok && elect_one()) mma_commit_pair(bar_acc + 8 * buf);
            }
            if (elect_one()) {
                if (!ok) fail(&abort_flag);
                mma_commit_pair(bar_drain);
            }
        }
        if (lane == 0) mbar_wait_drain(bar_drain, 0, kWaitLimitNs);  // (in both: the last thing that arrives here)
    } else if (warp >= kWarpEpilogue) {
        const int quarter = warp & 3, half = (warp - kWarpEpilogue) >> 2;
        const uint32_t at0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * (kBN / 2);
        const uint32_t buffer = sbase + kStages * kStageBytes + (warp - kWarpEpilogue) * kOutBytes;
        uint32_t local = 0;
        bool ok = true;
        for (int n = 0, t; (t = tile_of_turn(n, first, step)) < a.tiles; ++n, ++local) {
            const int buf = local & 1;
            if (!warp_wait(bar_acc + 8 * buf, (local >> 1) & 1, &abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const TileAt at = tile_at<kMode>(a, t);
            const Group& g = a.g[at.g];
            const int row = at.m0 + kBM * rank + 32 * quarter + lane;
#pragma unroll 1
            for (int c = 0; c < kBN / 2; c += 32) {
                const int j = at.n0 + half * (kBN / 2) + c;
                if (j >= g.cols || (kMode != kApply && j > row - lane)) break;
                uint32_t r[32];
                tmem_ld32(at0 + buf * kBN + c, r);
                tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                store32<kMode>(g, at.z, v, row, j, buffer);
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(bar_free + 8 * buf, 0));
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

// ------------------------------------------------------------------ small matrices
// Matrices with r <= 128 rows whose X fits the shared memory of up to eight CTAs: one kernel does the whole step. Each
// CTA of a matrix's group holds a slice of X's columns ([64-column block][R rows][128 bytes], R = 64 or 128; the
// 128-byte swizzle makes a block a K-major operand of the slice's X X^T and an MN-major one of B X), the CTAs add
// their parts of A in rank order, compute B each for itself and turn their slices to the next X in place. What
// bounds it: the passes over g, m and p at the start and end, then the five iterations' chain of products,
// exchanges and barriers (about 5 us each; one 16 x 1160 takes 34 us, 64 adapters of up to 64 x 2567 82).
constexpr int kSmallItems = 128, kSmallThreads = 512, kMostSmallSmem = 225 * 1024;
template <int R>
struct Small {  // R rows of X
    static constexpr int kMostBlocks = R == 64 ? 24 : 8;   // 64-column blocks of X that fit a CTA
    static constexpr int kSliceBlocks = R == 64 ? 9 : 8;   // of a CTA's slice, as long as eight CTAs are enough: two CTAs fit an SM
    static constexpr int kBlockBytes = R * 128;
    static constexpr int kABytes = R / 64 * 16384;         // A: 128 rows of R halves
    static constexpr int kPBytes = R == 64 ? 16384 : 65536;  // the CTA's part of A in fp32, then B
    static constexpr int kTile = R == 64 ? 128 : 256;       // columns of B X at a time, two such regions in TMEM
    static constexpr int kTmemCols = 2 * kTile;            // (64 rows: two CTAs an SM)
    // Never so little that CTAs of clusters would share an SM whose TMEM does not serve them all: one that waits for
    // TMEM while its cluster waits for it could wait forever. Two CTAs of 256 columns share one (80 KB each at least: no
    // third fits; the 8-bit product of few tokens likewise), one of 512 columns has it alone (beside 152 KB no 80 fit).
    static constexpr int kLeastSmem = (R == 64 ? 80 : 152) * 1024;
    // X's rests, half as many bytes, lie beside it where that costs no CTA its place on the SM, else in the workspace
    // (16 x 1160 34.9 us a call, 36.4 with them there; 64 adapters, half of them so, 84.0 and 86.0 with all).
    __host__ __device__ static constexpr bool rests_fit(int blocks) {
        return R == 64 ? blocks <= 6 || (blocks > kSliceBlocks && blocks <= 16) : blocks <= 5;
    }
    __host__ __device__ static constexpr int smem(int blocks) {
        const int need = blocks * kBlockBytes / 2 * (rests_fit(blocks) ? 3 : 2) + kABytes + kPBytes + 1024;
        return need > kLeastSmem ? need : kLeastSmem;
    }
    static_assert(512 / kTmemCols * kLeastSmem + 80 * 1024 > 228 * 1024, "");
    static_assert(R == 128 || (2 * smem(6) <= 225 * 1024 && 2 * smem(kSliceBlocks) <= 225 * 1024), "");
    static_assert(smem(R == 64 ? 16 : 5) <= kMostSmallSmem && smem(kMostBlocks) <= kMostSmallSmem, "");
};

struct SmallItem {
    void* p;
    float* master;
    const void* g;
    float* m;
    uint8_t* rest;          // the slices' rests in the workspace, where shared memory has no room (Small::rests_fit)
    int rows, cols, width;  // width: columns of a slice (a multiple of 64)
    Rates rate;
    bool g32;
};
struct SmallArgs {
    SmallItem item[kSmallItems];
    int n, ctas, iterations;  // ctas: of a matrix (a cluster)
    float a, b, c, mu, eps;
    bool nesterov;
    double lr;
    const float *grad_scale, *lr_dev;  // lr_dev: read instead of lr
};

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ double load_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

// A warp's turn at the slice: up to 256 neighbouring elements in memory (of one row of X, or, where the matrix is
// tall, anywhere in its columns), 8 a lane: four neighbours twice where rows are 16-byte aligned, else eight 32 apart.
constexpr int kDeep = 8, kUnit = 32 * kDeep;
template <bool kVec>
__device__ __forceinline__ int offset_of(int d, int lane) {
    return kVec ? 4 * lane + (d & 3) + 128 * (d >> 2) : lane + 32 * d;
}
template <bool kVec>
__device__ __forceinline__ void load_unit(float (&v)[kDeep], const void* g, bool fp32, long long at, int left, int lane) {
    if (kVec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = 4 * lane + 128 * h;
            float4 x = make_float4(0, 0, 0, 0);
            if (o + 4 <= left) {
                if (fp32) {
                    x = *reinterpret_cast<const float4*>(static_cast<const float*>(g) + at + o);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + at + o);
                    x = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
                }
            } else if (o < left) {  // (the slice's last elements)
                float* const y = &x.x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (o + j < left)
                        y[j] = fp32 ? static_cast<const float*>(g)[at + o + j]
                                    : __uint_as_float((uint32_t)static_cast<const uint16_t*>(g)[at + o + j] << 16);
            }
            v[4 * h] = x.x, v[4 * h + 1] = x.y, v[4 * h + 2] = x.z, v[4 * h + 3] = x.w;
        }
        return;
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        const int o = offset_of<kVec>(d, lane);
        v[d] = o >= left ? 0.0f
               : fp32    ? static_cast<const float*>(g)[at + o]
                         : __uint_as_float((uint32_t)static_cast<const uint16_t*>(g)[at + o] << 16);
    }
}
template <bool kVec>
__device__ __forceinline__ void store_unit(float* p, long long at, const float (&v)[kDeep], int left, int lane) {
    if (kVec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = 4 * lane + 128 * h;
            if (o + 4 <= left) {
                *reinterpret_cast<float4*>(p + at + o) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (o + j < left) p[at + o + j] = v[4 * h + j];
            }
        }
        return;
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        const int o = offset_of<kVec>(d, lane);
        if (o < left) p[at + o] = v[d];
    }
}
template <bool kVec>
__device__ __forceinline__ void store_unit_bf16(uint16_t* p, long long at, const float (&v)[kDeep], int left, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int o = 4 * lane + 128 * h;
        if (kVec && o + 4 <= left) {
            *reinterpret_cast<uint2*>(p + at + o) = make_uint2(pack_bf16(v[4 * h], v[4 * h + 1]), pack_bf16(v[4 * h + 2], v[4 * h + 3]));
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = offset_of<kVec>(4 * h + j, lane);
            if (e < left) p[at + e] = __bfloat16_as_ushort(__float2bfloat16_rn(v[4 * h + j]));
        }
    }
}

constexpr int kPiece = 2048;  // elements a prefetch takes
// The 16-byte pieces that lie within [p, p + bytes).
__device__ __forceinline__ void prefetch_l2(const void* p, long long bytes) {
    const uint64_t lo = (reinterpret_cast<uint64_t>(p) + 15) & ~15ull, hi = (reinterpret_cast<uint64_t>(p) + bytes) & ~15ull;
    if (hi > lo) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)(hi - lo)) : "memory");
}

struct Unit {
    long long at;  // first element
    int left;      // elements from there on
    int i, c;      // its place in X; tall: c alone counts, as an index
};
__device__ __forceinline__ Unit unit_of(int u, int per_row, int live, int r, int k, int col0, bool tall) {
    Unit x;
    if (tall) {
        x.i = 0;
        x.c = u * kUnit;
        x.at = (long long)col0 * r + x.c;
        x.left = live * r - x.c;
    } else {
        x.i = u / per_row;
        x.c = (u - x.i * per_row) * kUnit;
        x.at = (long long)x.i * k + col0 + x.c;
        x.left = live - x.c;
    }
    return x;
}

// What the passes over a slice need to know.
struct Slice {
    int per_row, units, live, r, k, col0, block_bytes;
    float inv_r;
    bool tall;
    int rows;  // of the memory: 64 or 128
    uint8_t *x, *rest;  // (rest: shared memory or the workspace)
    __device__ __forceinline__ Unit unit(int u) const { return unit_of(u, per_row, live, r, k, col0, tall); }
    // where X holds the element o of a tall matrix's unit
    __device__ __forceinline__ __half* tall_at(const Unit& u, int o) const {
        const int e = u.c + o, c = __float2int_rz(((float)e + 0.5f) * inv_r), i = e - c * r;  // (e / r, exact below 2^22)
        return reinterpret_cast<__half*>(x + (c >> 6) * block_bytes + i * 128 + ((((c & 63) >> 3) ^ (i & 7)) << 4) + (c & 7) * 2);
    }
    __device__ __forceinline__ void tall_put(const Unit& u, int o, __half h, uint8_t code) const {
        const int e = u.c + o, c = __float2int_rz(((float)e + 0.5f) * inv_r), i = e - c * r;
        *tall_at(u, o) = h;
        rests_at(c >> 4, i)[c & 15] = code;
    }
    // Where X holds the lane's four neighbours h (vectors), or its element d: a unit starts at a multiple of 256 columns.
    __device__ __forceinline__ uint2* four_at(const Unit& u, int h, int lane) const {
        return reinterpret_cast<uint2*>(x + ((u.c >> 6) + 2 * h + (lane >> 4)) * block_bytes + u.i * 128 +
                                        ((((lane & 15) >> 1) ^ (u.i & 7)) << 4) + (lane & 1) * 8);
    }
    __device__ __forceinline__ __half* one_at(const Unit& u, int d, int lane) const {
        return reinterpret_cast<__half*>(x + ((u.c >> 6) + (d >> 1)) * block_bytes + u.i * 128 +
                                         ((((lane >> 3) + 4 * (d & 1)) ^ (u.i & 7)) << 4) + (lane & 7) * 2);
    }
    // Where the rests of row i's 16 columns from 16 h on lie: a warp's 32 rows one behind the other.
    __device__ __forceinline__ uint8_t* rests_at(int h, int i) const { return rest + (h * rows + i) * 16; }
    // X = v * scale and its rests. (A row's slice ends at a multiple of 4 columns where there are vectors; X has room up to
    // a multiple of 64.)
    template <bool kVec>
    __device__ __forceinline__ void put(const Unit& u, const float (&v)[kDeep], float scale, int lane) const {
#pragma unroll
        for (int d = 0; d < kDeep; d += kVec ? 4 : 1) {
            const int o = offset_of<kVec>(d, lane);
            if (o >= u.left) continue;
            constexpr int kWide = kVec ? 4 : 1;
            __half2 h[kVec ? 2 : 1];
            uint32_t codes = 0;
#pragma unroll
            for (int j = 0; j < kWide; j += 2) {
                const float x0 = v[d + j] * scale, x1 = kVec ? v[(d + j + 1) % kDeep] * scale : 0.0f;
                h[j / 2] = __floats2half2_rn(x0, x1);
                codes |= rests2(x0, x1, h[j / 2], kRestScaleStart) << 8 * j;
            }
            if (tall) {
#pragma unroll
                for (int j = 0; j < kWide; ++j)
                    if (o + j < u.left) tall_put(u, o + j, j & 1 ? __high2half(h[j / 2]) : __low2half(h[j / 2]), (uint8_t)(codes >> 8 * j));
            } else if (kVec) {
                *four_at(u, d >> 2, lane) = make_uint2(*reinterpret_cast<const uint32_t*>(&h[0]), *reinterpret_cast<const uint32_t*>(&h[kVec ? 1 : 0]));
                *reinterpret_cast<uint32_t*>(rests_at((u.c + o) >> 4, u.i) + ((u.c + o) & 15)) = codes;
            } else {
                *one_at(u, d, lane) = __low2half(h[0]);
                rests_at((u.c + o) >> 4, u.i)[(u.c + o) & 15] = (uint8_t)codes;
            }
        }
    }
    template <bool kVec>
    __device__ __forceinline__ void get(const Unit& u, float (&v)[kDeep], int lane) const {
#pragma unroll
        for (int d = 0; d < kDeep; d += kVec ? 4 : 1) {
            const int o = offset_of<kVec>(d, lane);
#pragma unroll
            for (int j = 0; j < (kVec ? 4 : 1); ++j) v[d + j] = 0.0f;
            if (o >= u.left) continue;
            if (tall) {
#pragma unroll
                for (int j = 0; j < (kVec ? 4 : 1); ++j)
                    if (o + j < u.left) v[d + j] = __half2float(*tall_at(u, o + j));
            } else if (kVec) {
                const uint2 w = *four_at(u, d >> 2, lane);
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), q = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
                v[d] = p.x, v[(d + 1) % kDeep] = p.y, v[(d + 2) % kDeep] = q.x, v[(d + 3) % kDeep] = q.y;
            } else {
                v[d] = __half2float(*one_at(u, d, lane));
            }
        }
    }
};

// The power of two that brings `top` to 2^8 (fp16 then has 2^22 below it as normal numbers, and values up to 2^12 find
// room for their rests); 0 and what is not finite: 1.
__device__ __forceinline__ float x_scale(float top) {
    const int e = (int)(__float_as_uint(top) >> 23);
    return top > 0.0f && e < 255 ? __uint_as_float((uint32_t)min(max(127 + 8 - (e - 127), 1), 254) << 23) : 1.0f;
}

// u of one unit: the new momentum is written (kMomentum), or was and is read again.
template <bool kVec, bool kMomentum>
__device__ __forceinline__ void update_of(float (&u)[kDeep], const SmallItem& it, const SmallArgs& a, const Unit& x, float f, int lane) {
    load_unit<kVec>(u, it.g, it.g32, x.at, x.left, lane);
    if (it.m == nullptr) return;
    float m[kDeep];
    load_unit<kVec>(m, it.m, true, x.at, x.left, lane);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        const float g = u[d] * f;
        if (kMomentum) m[d] = fmaf(a.mu, m[d], g);
        u[d] = a.nesterov ? fmaf(a.mu, m[d], g) : m[d];
    }
    if (kMomentum) store_unit<kVec>(it.m, x.at, m, x.left, lane);
}
__device__ __forceinline__ float block_top(float top, float* sums) {  // over the CTA's threads
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = top;
    __syncthreads();
    top = sums[threadIdx.x % (kSmallThreads / 32)];
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    return top;
}

// One read of the slice: momentum, sum of u's squares, X = u * scale. The scale comes from the warps' first units; if
// some value does not fit it after all, X is written again with one that fits (from the momentum as it is now).
template <bool kVec>
__device__ __forceinline__ float read_slice(const SmallItem& it, const SmallArgs& a, const Slice& s, float f, float* sums, float& sq) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kWarps = kSmallThreads / 32;
    float u[kDeep], top = 0.0f;
    auto look = [&]() {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            sq = fmaf(u[d], u[d], sq);
            top = fmaxf(top, fabsf(u[d]));
        }
    };
    sq = 0.0f;
    Unit x = s.unit(min(warp, s.units - 1));
    if (warp < s.units) {
        update_of<kVec, true>(u, it, a, x, f, lane);
        look();
    }
    float scale = x_scale(block_top(top, sums));
    if (warp < s.units) s.put<kVec>(x, u, scale, lane);
    for (int n = warp + kWarps; n < s.units; n += kWarps) {
        x = s.unit(n);
        update_of<kVec, true>(u, it, a, x, f, lane);
        look();
        s.put<kVec>(x, u, scale, lane);
    }
    top = block_top(top, sums);
    if (top * scale < 4096.0f && (top * scale >= 1.0f || top == 0.0f)) return scale;
    scale = x_scale(top);
    for (int n = warp; n < s.units; n += kWarps) {
        x = s.unit(n);
        update_of<kVec, false>(u, it, a, x, f, lane);
        s.put<kVec>(x, u, scale, lane);
    }
    return scale;
}

// p -= decay p + rate X, or p = X
template <bool kVec>
__device__ __forceinline__ void write_slice(const SmallItem& it, const Slice& s, float rate, float decay) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* const w32 = it.master != nullptr ? it.master : static_cast<float*>(it.p);
    for (int n = warp; n < s.units; n += kSmallThreads / 32) {
        const Unit x = s.unit(n);
        float w[kDeep];
        float v[kDeep];
        if (it.m != nullptr) load_unit<kVec>(w, w32, true, x.at, x.left, lane);
        s.get<kVec>(x, v, lane);
#pragma unroll
        for (int d = 0; d < kDeep; ++d) w[d] = it.m != nullptr ? w[d] - fmaf(decay, w[d], rate * v[d]) : v[d];
        if (it.m != nullptr) store_unit<kVec>(w32, x.at, w, x.left, lane);
        if (it.m == nullptr || it.master != nullptr) store_unit_bf16<kVec>(static_cast<uint16_t*>(it.p), x.at, w, x.left, lane);
    }
}

template <int R>
__global__ void __launch_bounds__(kSmallThreads, R == 64 ? 2 : 1) muon_small_kernel(const __grid_constant__ SmallArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2];  // products: two regions of TMEM take turns
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ float s_sums[kSmallThreads / 32], s_inv, s_rates[2];
    __shared__ __align__(16) float s_group[8];  // X's sum of squares, each CTA's
    __shared__ __align__(8) double s_part;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const float f = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    // The step's other launches of small matrices may run beside this one: they share nothing. Each waits for the one
    // before it at its end, so that the last one's end is the end of all.
    asm volatile("griddepcontrol.launch_dependents;");
    const int ctas = a.ctas, rank = blockIdx.x % ctas;
    const SmallItem& it = a.item[blockIdx.x / ctas];
    if (!(fabsf(f) < INFINITY)) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const bool tall = it.rows > it.cols;
    const int r = tall ? it.cols : it.rows, k = tall ? it.rows : it.cols;
    const int col0 = rank * it.width, live = max(0, min(it.width, k - col0));
    const int blocks = it.width / 64;
    constexpr int block_bytes = Small<R>::kBlockBytes, kTile = Small<R>::kTile;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sx = sbase, sa = sbase + blocks * block_bytes, sb = sa + Small<R>::kABytes, sp = sb;
    uint8_t* const generic = smem_raw + (sbase - smem_u32(smem_raw));
    uint8_t* const rest = Small<R>::rests_fit(blocks) ? generic + (sb - sbase) + Small<R>::kPBytes
                                                      : it.rest + (long long)rank * blocks * (block_bytes / 2);
    const uint32_t bar_mma = smem_u32(&bars[0]);

    if (tid == 0) {
        abort_flag = 0;
        for (int w = ctas; w < 8; ++w) s_group[w] = 0.0f;
        mbar_init(bar_mma, 1);
        mbar_init(bar_mma + 8, 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_slot), Small<R>::kTmemCols);
        tmem_relinquish();
    }
    for (int i = tid; i < blocks * block_bytes / 16; i += kSmallThreads) {
        reinterpret_cast<uint4*>(generic)[i] = make_uint4(0, 0, 0, 0);
        if (i & 1) reinterpret_cast<uint4*>(rest)[i >> 1] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    uint32_t mma_phase[2] = {0, 0};
    auto bounded = [&](bool ok) {
        if (!ok) fail(&abort_flag);
    };
    auto group_sync = [&]() {
        if (ctas > 1)
            cluster_sync_all();
        else
            __syncthreads();
    };
    auto mma_wait = [&](int w) {
        bounded(mbar_wait(bar_mma + 8 * w, mma_phase[w], &abort_flag, kWaitLimitNs));
        mma_phase[w] ^= 1;
        tc_fence_after();
    };
    auto publish = [&]() {  // shared memory written by every thread, TMEM read by every thread: before the next products
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // byte offset of row i, 16-byte chunk q of a swizzled block of 128-byte rows
    auto chunk_at = [&](int i, int q) { return i * 128 + ((q ^ (i & 7)) << 4); };

    // ---- momentum, norm, X
    // What the passes read is fetched to L2 first, in a few instructions: X leaves little of the SM's memory to the
    // cache that plain loads in flight need.
    const float* const w32 = it.master != nullptr ? it.master : static_cast<const float*>(it.p);
    auto fetch = [&](bool weights) {
        const int es = it.g32 ? 4 : 2;
        const long long run = tall ? (long long)live * r : live, base = tall ? (long long)col0 * r : col0;
        const int runs = tall ? 1 : r, pieces = (int)((run + kPiece - 1) / kPiece);
        for (int e = tid; e < runs * pieces; e += kSmallThreads) {
            const int i = e / pieces;
            const long long from = base + (long long)i * k + (long long)(e - i * pieces) * kPiece;
            const long long n = min((long long)kPiece, run - (long long)(e - i * pieces) * kPiece);
            if (!weights) prefetch_l2(static_cast<const uint8_t*>(it.g) + from * es, n * es);
            if (it.m != nullptr) prefetch_l2(weights ? w32 + from : it.m + from, n * 4);
        }
    };
    fetch(false);
    Slice slice;
    slice.per_row = max(1, (live + kUnit - 1) / kUnit);
    slice.units = tall ? (live * r + kUnit - 1) / kUnit : live > 0 ? r * slice.per_row : 0;
    slice.live = live;
    slice.r = r;
    slice.inv_r = 1.0f / (float)r;
    slice.k = k;
    slice.col0 = col0;
    slice.block_bytes = block_bytes;
    slice.tall = tall;
    slice.x = generic;
    slice.rows = R;
    slice.rest = rest;
    const bool vec = tall || k % 4 == 0;  // (slices start at multiples of 64 columns)
    float sq;
    const float up = vec ? read_slice<true>(it, a, slice, f, s_sums, sq) : read_slice<false>(it, a, slice, f, s_sums, sq);
    __syncthreads();
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, w);
    if (lane == 0) s_sums[warp] = sq;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < kSmallThreads / 32; ++w) s += (double)s_sums[w];
        s_part = s;
    }
    if (tid == 32) it.rate.get(a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr, s_rates[0], s_rates[1]);
    if (it.m != nullptr) fetch(true);  // (what the last pass reads)
    group_sync();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < ctas; ++w) s += ctas == 1 ? s_part : load_cluster_f64(map_rank(smem_u32(&s_part), w));
        s_inv = 1.0f / (norm_of(s) + a.eps);
    }
    publish();

    // ---- iterations
    const int quarter = warp & 3, group = warp >> 2;  // a warp's 32 rows, and its quarter of the columns
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    constexpr uint32_t idesc_r = idesc_f16(128, R, false);
    constexpr int kOwn = R / 4;                      // columns of A and B a warp has
    constexpr uint32_t kPolyCol = R;                 // (the regions of B X lie over A's and B's)
    float scale = s_inv / up;  // X is what is stored times this, until the first iteration's end
    // X's squares, a thread's part each, lie where nothing is read or written from an iteration's end to its next barrier
    float* const squares = reinterpret_cast<float*>(generic + ((ctas == 1 ? sb : sa) - sbase));
    const Poly poly{a.a, a.b, a.c};
    const float rest_share = r == 1 ? 1.0f : r < 4 ? 0.0f : 0.25f;
    float shift = 1.0f / (float)r;  // the mean of A's diagonal: X's sum of squares (1 at first) a row
    for (int n = 0; n < a.iterations; ++n) {
        if (warp == 0) {  // the slice's part of X X^T
            const uint64_t x0 = sdesc_sw128(sx, 16, 1024);
            for (int j = 0; j < blocks; ++j) {
                const uint64_t d = x0 + j * (block_bytes >> 4);
                if (elect_one())
#pragma unroll
                    for (int q = 0; q < 4; ++q) mma_ss(tmem, d + 2 * q, d + 2 * q, idesc_r, j > 0 || q > 0 ? 1u : 0u);
            }
            if (elect_one()) mma_commit(bar_mma);
        }
        if (n > 0 && (ctas == 1 || warp == 1)) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kSmallThreads; w += 32) s += squares[w + lane];
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            if (ctas == 1)
                shift = s * slice.inv_r;
            else if (lane < ctas)  // (read between the iteration's two barriers, written after the last one's)
                store_cluster(map_rank(smem_u32(&s_group[rank]), lane), s);
        }
        mma_wait(0);
        if (row < R) {
#pragma unroll
            for (int c = group * kOwn; c < group * kOwn + kOwn; c += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + lanes + c, v);
                tmem_ld_wait();
                const auto part = [&](int j) { return __uint_as_float(v[j]) * scale * scale - (ctas == 1 && c + j == row ? shift : 0.0f); };
                if (ctas == 1) {  // all of D
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int q = c / 8 + h;
                        *reinterpret_cast<uint4*>(generic + (sa - sbase) + (q >> 3) * 16384 + chunk_at(row, q & 7)) =
                            make_uint4(pack_half(part(8 * h), part(8 * h + 1)), pack_half(part(8 * h + 2), part(8 * h + 3)),
                                       pack_half(part(8 * h + 4), part(8 * h + 5)), pack_half(part(8 * h + 6), part(8 * h + 7)));
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sp + row * R * 4 + (((c / 4 + q) ^ (row & 7)) << 4)),
                                     "f"(part(4 * q)), "f"(part(4 * q + 1)), "f"(part(4 * q + 2)), "f"(part(4 * q + 3))
                                     : "memory");
                }
            }
        }
        if (ctas > 1) {
            tc_fence_before();
            group_sync();
            if (n > 0) {
                const float4 p = *reinterpret_cast<const float4*>(s_group), q = *reinterpret_cast<const float4*>(s_group + 4);
                shift = ((p.x + p.y) + (p.z + p.w) + ((q.x + q.y) + (q.z + q.w))) * slice.inv_r;
            }
            // this CTA's rows of D, the parts in rank order, to every CTA of the group
            const int share = R / ctas, row0 = rank * share;
            for (int e = tid; e < share * (R / 4); e += kSmallThreads) {
                const int i = row0 + e / (R / 4), q = e % (R / 4);
                const uint32_t at = sp + i * R * 4 + ((q ^ (i & 7)) << 4);
                float4 v = make_float4(0, 0, 0, 0);
                for (int w = 0; w < ctas; ++w) {
                    const float4 t = load_cluster(map_rank(at, w));
                    v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
                }
                if (i >> 2 == q) (i & 2 ? i & 1 ? v.w : v.z : i & 1 ? v.y : v.x) -= shift;
                const uint32_t to = sa + (q >> 4) * 16384 + chunk_at(i, (q & 15) >> 1) + (q & 1) * 8;
                const uint32_t lo = pack_half(v.x, v.y), hi = pack_half(v.z, v.w);
                for (int w = 0; w < ctas; ++w)
                    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(map_rank(to, w)), "r"(lo), "r"(hi) : "memory");
            }
            group_sync();
        }
        publish();
        if (warp == 0) {  // D D
            const uint64_t a0 = sdesc_sw128(sa, 16, 1024);
#pragma unroll
            for (int h = 0; h < R / 64; ++h) {
                const uint64_t d = a0 + h * (16384 >> 4);
                if (elect_one())
#pragma unroll
                    for (int q = 0; q < 4; ++q) mma_ss(tmem + kPolyCol, d + 2 * q, d + 2 * q, idesc_r, h > 0 || q > 0 ? 1u : 0u);
            }
            if (elect_one()) mma_commit(bar_mma);
        }
        mma_wait(0);
        if (row < R) {
#pragma unroll
            for (int c = group * kOwn; c < group * kOwn + kOwn; c += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + kPolyCol + lanes + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = c / 8 + h, off = (q >> 3) * 16384 + chunk_at(row, q & 7);
                    const uint4 w = *reinterpret_cast<const uint4*>(generic + (sa - sbase) + off);
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
                        y[j] = pack_half(fmaf(poly.of_d(shift), d.x, a.c * __uint_as_float(v[8 * h + 2 * j])),
                                         fmaf(poly.of_d(shift), d.y, a.c * __uint_as_float(v[8 * h + 2 * j + 1])));
                    }
                    const uint4 b = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(generic + (sb - sbase) + off) = b;
                    if (R == 64)  // once more in the rows from 64 on, so that the other half of TMEM's lanes holds B X too
                        *reinterpret_cast<uint4*>(generic + (sb - sbase) + off + 64 * 128) = b;
                }
            }
        }
        publish();
        // X = a X + B X (the coefficients of D's polynomial), kTile columns at a time in two regions of TMEM
        constexpr int kTileBlocks = kTile / 64;
        const int tiles = (blocks + kTileBlocks - 1) / kTileBlocks;
        auto issue = [&](int t) {
            if (warp != 0) return;
            const uint32_t idesc = idesc_f16(128, 64 * min(kTileBlocks, blocks - kTileBlocks * t), true);
            const uint64_t b0 = sdesc_sw128(sb, 16, 1024);
            const uint64_t x0 = sdesc_sw128(sx + kTileBlocks * t * block_bytes, block_bytes, 1024);
#pragma unroll
            for (int h = 0; h < R / 64; ++h)
                if (elect_one())
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_ss(tmem + kTile * (t & 1), b0 + h * (16384 >> 4) + 2 * q, x0 + (4 * h + q) * (2048 >> 4), idesc,
                               h > 0 || q > 0 ? 1u : 0u);
            if (elect_one()) mma_commit(bar_mma + 8 * (t & 1));
        };
        issue(0);
        if (tiles > 1) issue(1);
        const float of_x = poly.of_x(shift) * scale;
        // a warp's columns of a tile: a quarter of it; where the lanes from 64 on hold the same rows again, half of that
        const int i = R == 64 ? row & 63 : row, own0 = R == 64 ? group * 32 + (quarter >> 1) * 16 : group * 64;
        const float of_rest = (n + 1 < kRests ? poly.of_x(shift * rest_share) * scale : of_x) / (n == 0 ? kRestScaleStart : kRestScale);
        const uint64_t of_x2 = f2_pack(of_x, of_x), scale2 = f2_pack(scale, scale), of_rest2 = f2_pack(of_rest, of_rest);
        __half2 square = __float2half2_rn(0.0f);
        auto turn = [&](auto reads, auto writes) {  // (a form each: a branch within the loop costs every iteration)
            constexpr bool kRead = decltype(reads)::value, kWrite = decltype(writes)::value;
            for (int t = 0; t < tiles; ++t) {
                mma_wait(t & 1);
#pragma unroll
                for (int c = own0; c < own0 + (R == 64 ? 16 : 64); c += 16) {
                    const int block = kTileBlocks * t + (c >> 6);
                    if (block >= blocks) break;
                    // (everything is read before anything is written)
                    uint4* const low = reinterpret_cast<uint4*>(slice.rests_at((kTile * t + c) >> 4, i));
                    uint4 rests = make_uint4(0, 0, 0, 0);
                    if (kRead) rests = *low;
                    uint4* const at0 = reinterpret_cast<uint4*>(generic + block * block_bytes + chunk_at(i, (c & 63) >> 3));
                    uint4* const at1 = reinterpret_cast<uint4*>(generic + block * block_bytes + chunk_at(i, ((c & 63) >> 3) + 1));
                    const uint4 w0 = *at0, w1 = *at1;
                    uint32_t v[16];
                    tmem_ld16(tmem + kTile * (t & 1) + lanes + c, v);
                    tmem_ld_wait();
                    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                    uint64_t x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                        x[j] = fma_f2(of_x2, f2_pack(y.x, y.y), mul_f2(scale2, f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]))));
                    }
                    if (kRead) {
                        const uint32_t l[4] = {rests.x, rests.y, rests.z, rests.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 y = rest_values(l[j >> 1] >> 16 * (j & 1));
                            x[j] = fma_f2(of_rest2, f2_pack(y.x, y.y), x[j]);
                        }
                    }
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x0, x1;
                        f2_unpack(x[j], x0, x1);
                        const __half2 y2 = __floats2half2_rn(x0, x1);
                        square = __hfma2(y2, y2, square);  // (fp16 is enough for where to shift)
                        o[j] = *reinterpret_cast<const uint32_t*>(&y2);
                    }
                    *at0 = make_uint4(o[0], o[1], o[2], o[3]);
                    *at1 = make_uint4(o[4], o[5], o[6], o[7]);
                    if (kWrite) {
                        uint32_t l[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < 8; ++j) l[j >> 1] |= rests2(x[j], *reinterpret_cast<const __half2*>(&o[j]), kRestScale) << 16 * (j & 1);
                        *low = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                }
                if (t + 2 < tiles) {  // (the tile is read out)
                    tc_fence_before();
                    __syncthreads();
                    tc_fence_after();
                    issue(t + 2);
                }
            }
        };
        if (n + 1 < kRests)
            turn(std::true_type{}, std::true_type{});
        else if (n < kRests)
            turn(std::true_type{}, std::false_type{});
        else
            turn(std::false_type{}, std::false_type{});
        squares[tid] = __low2float(square) + __high2float(square);
        publish();
        scale = 1.0f;
    }

    // ---- the weights, or X itself
    const float rate = s_rates[0], decay = s_rates[1];
    if (vec)
        write_slice<true>(it, slice, rate, decay);
    else
        write_slice<false>(it, slice, rate, decay);
    tc_fence_before();
    group_sync();  // nobody leaves while another reads its memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Small<R>::kTmemCols);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ host
size_t up(size_t x, size_t k) { return (x + k - 1) / k * k; }

// Where a list's matrices lie in the workspace.
struct Size {
    int r, k, ld, ldr, ld_rest, count;  // r <= k; rows of X, of A and B, of the rests: elements apart
    size_t x[2], b, rest;              // byte offsets: X twice (read and written in turn; A lies in the one that is to be
                                       // written next), B, the rests
};
struct Plan {
    std::vector<Size> sizes;
    std::vector<int> of, z, parts;     // a matrix's size, its place among them, its partial sums
    std::vector<long long> chunk;
    std::vector<size_t> part;          // byte offset of its partial sums; small matrices: of their rests
    size_t bytes = 0;
};

// CTAs of a small matrix's group, 0 for one that takes the products of whole launches: the fewest (a power of two)
// with slices of 576 (above 64 rows: 512) columns at most, or eight whose shared memory holds X. By its size alone, so that the sums over
// its columns have one order in every list.
int small_ctas(const rlk_muon_matrix& t) {
    const long long r = t.rows < t.cols ? t.rows : t.cols, k = t.rows < t.cols ? t.cols : t.rows;
    if (r > 128) return 0;
    int n = 1;
    while (n < 8 && k > n * 64LL * (r <= 64 ? Small<64>::kSliceBlocks : Small<128>::kSliceBlocks)) n *= 2;
    return k <= n * 64LL * (r <= 64 ? Small<64>::kMostBlocks : Small<128>::kMostBlocks) ? n : 0;
}

// Columns of a CTA's slice, and bytes of the rests that find no room in shared memory.
int small_width(const rlk_muon_matrix& t, int ctas) {
    const long long k = t.rows < t.cols ? t.cols : t.rows;
    return (int)up((k + ctas - 1) / ctas, 64);
}
size_t small_rests(const rlk_muon_matrix& t, int ctas) {
    const int r = (int)(t.rows < t.cols ? t.rows : t.cols), width = small_width(t, ctas);
    if (r <= 64 ? Small<64>::rests_fit(width / 64) : Small<128>::rests_fit(width / 64)) return 0;
    return (size_t)ctas * width * (r <= 64 ? 64 : 128);
}

void plan_of(const rlk_muon_matrix* t, int n, Plan& p) {
    p.of.assign(n, -1);
    p.z.assign(n, 0);
    p.parts.assign(n, 0);
    p.chunk.assign(n, 0);
    p.part.assign(n, 0);
    std::map<std::pair<int, int>, int> known;
    for (int i = 0; i < n; ++i) {
        if (t[i].rows == 0 || t[i].cols == 0) continue;
        if (const int ctas = small_ctas(t[i])) {
            p.bytes = up(p.bytes, 16);
            p.part[i] = p.bytes;
            p.bytes += small_rests(t[i], ctas);
            continue;
        }
        const int r = (int)(t[i].rows < t[i].cols ? t[i].rows : t[i].cols), k = (int)(t[i].rows < t[i].cols ? t[i].cols : t[i].rows);
        const int s = known.emplace(std::make_pair(r, k), (int)p.sizes.size()).first->second;
        if (s == (int)p.sizes.size()) p.sizes.push_back(Size{r, k, (int)up(k, 8), (int)up(r, 8), (int)up(k, 16), 0, {0, 0}, 0, 0});
        p.of[i] = s;
        p.z[i] = p.sizes[s].count++;
        const long long e = t[i].rows * t[i].cols;
        long long chunk = (e + kMaxPartials - 1) / kMaxPartials;
        chunk = (long long)up(chunk < kMinChunk ? kMinChunk : chunk, 4 * kPassThreads);
        p.chunk[i] = chunk;
        p.parts[i] = (int)((e + chunk - 1) / chunk);
        p.bytes = up(p.bytes, sizeof(double));
        p.part[i] = p.bytes;
        p.bytes += sizeof(double) * (p.parts[i] + 1);  // (and its rates)
    }
    for (Size& s : p.sizes) {
        auto take = [&](size_t bytes) {
            p.bytes = up(p.bytes, 256);
            const size_t at = p.bytes;
            p.bytes += bytes;
            return at;
        };
        for (size_t& x : s.x) x = take((size_t)s.count * s.r * s.ld * 2);
        s.b = take((size_t)s.count * s.r * s.ldr * 2);
        s.rest = take((size_t)s.count * s.r * s.ld_rest);
    }
}

bool half_map(CUtensorMap* m, const void* base, int cols, int rows, int count, int ld, int box_rows, bool out = false) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)rows * ld * 2};
    const cuuint32_t box[3] = {out ? 32u : 64u, (cuuint32_t)box_rows, 1};
    return tmap::encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box,
                        out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kMode>
cudaError_t launch_product(GemmArgs& a, int pairs, cudaStream_t s) {
    a.tiles = 0;
    for (int g = 0; g < a.n; ++g) {
        Group& d = a.g[g];
        const int blocks = (d.rows + 2 * kBM - 1) / (2 * kBM);
        d.per = kMode == kApply ? blocks * ((d.cols + kBN - 1) / kBN) : blocks * (blocks + 1) / 2;
        d.tile0 = a.tiles;
        a.tiles += d.per * d.count;
    }
    cudaError_t e = cudaFuncSetAttribute(muon_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(2u * (unsigned)(a.tiles < pairs ? a.tiles : pairs));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kSmemBytes;
    c.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = 1;
    const int id = kMode == kGram ? kKMuonGram : kMode == kPoly ? kKMuonPoly : kKMuonApply;
    timing_begin(id, s);
    e = cudaLaunchKernelEx(&c, muon_gemm_kernel<kMode>, a);
    timing_end(id, s);
    return e;
}

// Clusters of two that fit the device at once: more would wait for the first to end.
cudaError_t pairs_of(int* pairs) {
    static std::atomic<int> fit[64];
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*pairs = fit[dev].load()) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(muon_gemm_kernel<kApply>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(2 * (sms / 2));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kSmemBytes;
    e = cudaOccupancyMaxActiveClusters(pairs, muon_gemm_kernel<kApply>, &c);
    if (e == cudaSuccess && *pairs < 1) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess && dev < 64) fit[dev].store(*pairs);
    return e;
}

// One pass over the list: kItems matrices a launch, those with 16-byte aligned rows in launches of their own where the
// pass makes a difference between them.
template <typename Blocks, typename Launch>
cudaError_t pass(const std::vector<Item>& items, PassArgs& a, bool apart, Blocks blocks_of, Launch launch) {
    for (int vec = apart ? 0 : 1; vec < 2; ++vec) {
        a.n = 0;
        int blocks = 0;
        for (size_t i = 0; i <= items.size(); ++i) {
            if (a.n > 0 && (a.n == kItems || i == items.size())) {
                launch(blocks, vec == 1);
                const cudaError_t e = cudaGetLastError();
                if (e != cudaSuccess) return e;
                a.n = blocks = 0;
            }
            if (i == items.size() || (apart && (items[i].cols % 8 == 0) != (vec == 1))) continue;
            a.item[a.n] = items[i];
            a.item[a.n++].block0 = blocks;
            blocks += blocks_of(items[i]);
        }
    }
    return cudaSuccess;
}

float start_of(long long r) { return (float)exp2(floor(0.5 * log2((double)r))); }

Rates rates_of(const rlk_muon_matrix& d, const rlk_muon_args& q) {
    return Rates{d.lr_scale, d.weight_decay, q.update_rms, sqrt((double)(d.rows > d.cols ? d.rows : d.cols))};
}

// The small matrices of up to R rows (and more than 64, if R is 128), those of one number of CTAs a launch; `more`: a
// launch of them came before, and this one may run beside it.
template <int R>
cudaError_t run_small(const rlk_muon_matrix* t, int n, const rlk_muon_args& q, bool step, const Plan& plan, uint8_t* ws, bool& more,
                      cudaStream_t s) {
    SmallArgs a;
    a.iterations = q.iterations;
    a.a = (float)q.a;
    a.b = (float)q.b;
    a.c = (float)q.c;
    a.mu = (float)q.momentum;
    a.eps = (float)q.eps;
    a.nesterov = q.nesterov != 0;
    a.grad_scale = step ? q.grad_scale : nullptr;
    a.lr = step ? q.lr : 0.0;
    a.lr_dev = step ? q.lr_dev : nullptr;
    int smem = 0;  // what the matrix that needs most takes
    auto launch = [&]() {
        cudaError_t e = cudaFuncSetAttribute(muon_small_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMostSmallSmem);
        // (all of it for shared memory: two CTAs an SM)
        if (e == cudaSuccess) e = cudaFuncSetAttribute(muon_small_kernel<R>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3((unsigned)(a.n * a.ctas));
        c.blockDim = dim3(kSmallThreads);
        c.dynamicSmemBytes = smem;
        c.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = a.ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = more ? 2 : 1;
        timing_begin(kKMuonSmall, s);
        e = cudaLaunchKernelEx(&c, muon_small_kernel<R>, a);
        timing_end(kKMuonSmall, s);
        more = true;
        return e;
    };
    for (a.ctas = 8; a.ctas > 0; a.ctas /= 2) {
        a.n = smem = 0;
        for (int i = 0; i <= n; ++i) {
            if (a.n > 0 && (i == n || a.n == kSmallItems)) {
                const cudaError_t e = launch();
                if (e != cudaSuccess) return e;
                a.n = smem = 0;
            }
            if (i == n) break;
            const rlk_muon_matrix& d = t[i];
            const long long r = d.rows < d.cols ? d.rows : d.cols;
            if (r == 0 || (r <= 64) != (R == 64) || small_ctas(d) != a.ctas) continue;
            SmallItem& it = a.item[a.n++];
            it.p = d.p;
            it.master = step ? d.master : nullptr;
            it.g = d.g;
            it.m = step ? d.m : nullptr;
            it.rows = (int)d.rows;
            it.cols = (int)d.cols;
            it.width = small_width(d, a.ctas);
            it.rest = ws + plan.part[i];
            it.rate = rates_of(d, q);
            it.g32 = d.g_dtype == RLK_FP32;
            if (Small<R>::smem(it.width / 64) > smem) smem = Small<R>::smem(it.width / 64);
        }
    }
    return cudaSuccess;
}

cudaError_t run(const rlk_muon_matrix* t, int n, const rlk_muon_args& q, bool step, void* workspace, cudaStream_t s) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Plan plan;
    plan_of(t, n, plan);
    bool more = false;
    for (const auto small : {run_small<64>, run_small<128>}) {
        const cudaError_t e = small(t, n, q, step, plan, ws, more, s);
        if (e != cudaSuccess) return e;
    }
    if (plan.sizes.empty()) return cudaSuccess;
    int pairs = 0;
    cudaError_t e = pairs_of(&pairs);
    if (e != cudaSuccess) return e;
    std::vector<Item> items;
    std::vector<float> start(plan.sizes.size());
    for (size_t i = 0; i < plan.sizes.size(); ++i) start[i] = start_of(plan.sizes[i].r);
    for (int i = 0; i < n; ++i) {
        if (plan.of[i] < 0) continue;
        const rlk_muon_matrix& d = t[i];
        const Size& z = plan.sizes[plan.of[i]];
        Item it{};
        it.p = d.p;
        it.master = step ? d.master : nullptr;
        it.g = d.g;
        it.m = step ? d.m : nullptr;
        it.x = reinterpret_cast<__half*>(ws + z.x[0]) + (size_t)plan.z[i] * z.r * z.ld;
        it.rest = ws + z.rest + (size_t)plan.z[i] * z.r * z.ld_rest;
        it.ld_rest = z.ld_rest;
        it.part = reinterpret_cast<double*>(ws + plan.part[i]);
        it.n = d.rows * d.cols;
        it.chunk = plan.chunk[i];
        it.rows = (int)d.rows;
        it.cols = (int)d.cols;
        it.ld = z.ld;
        it.parts = plan.parts[i];
        it.start = start[plan.of[i]];
        it.rate = rates_of(d, q);
        it.rates = reinterpret_cast<float*>(ws + plan.part[i] + sizeof(double) * plan.parts[i]);
        it.g32 = d.g_dtype == RLK_FP32;
        items.push_back(it);
    }
    if (items.empty()) return cudaSuccess;
    PassArgs a;
    a.mu = (float)q.momentum;
    a.eps = (float)q.eps;
    a.nesterov = q.nesterov != 0;
    a.grad_scale = step ? q.grad_scale : nullptr;
    a.lr = step ? q.lr : 0.0;
    a.lr_dev = step ? q.lr_dev : nullptr;
    auto tiles = [](const Item& it) { return ((it.rows + kSide - 1) / kSide) * ((it.cols + kSide - 1) / kSide); };
    e = pass(items, a, false, [](const Item& it) { return it.parts; }, [&](int blocks, bool) {
        timing_begin(kKMuonMomentum, s);
        muon_momentum_kernel<<<blocks, kPassThreads, 0, s>>>(a);
        timing_end(kKMuonMomentum, s);
    });
    if (e == cudaSuccess) e = pass(items, a, true, tiles, [&](int blocks, bool vec) {
        timing_begin(kKMuonStart, s);
        (vec ? muon_start_kernel<true> : muon_start_kernel<false>)<<<blocks, kPassThreads, 0, s>>>(a);
        timing_end(kKMuonStart, s);
    });
    if (e != cudaSuccess) return e;
    for (size_t g0 = 0; g0 < plan.sizes.size(); g0 += kGroups) {
        const int ng = (int)(plan.sizes.size() - g0 < kGroups ? plan.sizes.size() - g0 : kGroups);
        // X as the operand of 128 rows (gram) and of 256 columns (apply), both buffers; A; B
        CUtensorMap x_rows[kGroups][2], x_cols[kGroups][2], x_out[kGroups][2], map_a[kGroups][2], a_out[kGroups][2], map_b[kGroups], b_out[kGroups];
        for (int g = 0; g < ng; ++g) {
            const Size& z = plan.sizes[g0 + g];
            bool ok = half_map(&map_b[g], ws + z.b, z.r, z.r, z.count, z.ldr, 128) &&
                      half_map(&b_out[g], ws + z.b, z.r, z.r, z.count, z.ldr, 32, true);
            for (int i = 0; i < 2; ++i)
                ok = ok && half_map(&x_rows[g][i], ws + z.x[i], z.k, z.r, z.count, z.ld, 128) &&
                     half_map(&x_cols[g][i], ws + z.x[i], z.k, z.r, z.count, z.ld, 64) &&
                     half_map(&x_out[g][i], ws + z.x[i], z.k, z.r, z.count, z.ld, 32, true) &&
                     half_map(&map_a[g][i], ws + z.x[i], z.r, z.r, z.count, z.ldr, 128) &&
                     half_map(&a_out[g][i], ws + z.x[i], z.r, z.r, z.count, z.ldr, 32, true);
            if (!ok) return cudaErrorInvalidValue;
        }
        const Poly poly{(float)q.a, (float)q.b, (float)q.c};
        float shift[kGroups], square[kGroups];
        for (int g = 0; g < ng; ++g) square[g] = kSpread / (float)plan.sizes[g0 + g].r;
        for (int i = 0; i < q.iterations; ++i) {
            for (int g = 0; g < ng; ++g) {
                const float p = poly.of_x(square[g]);
                shift[g] = fminf(square[g], 1.0f);  // (1 for a NaN)
                square[g] *= p * p;
            }
            for (int mode = kGram; mode <= kApply; ++mode) {
                GemmArgs ga;
                ga.n = ng;
                int order[kGroups];  // the longest sums first
                for (int g = 0; g < ng; ++g) order[g] = g;
                auto length = [&](int g) { return mode == kGram ? plan.sizes[g0 + g].k : plan.sizes[g0 + g].r; };
                std::stable_sort(order, order + ng, [&](int x, int y) { return length(x) > length(y); });
                for (int n_g = 0; n_g < ng; ++n_g) {
                    const int g = order[n_g];
                    const Size& z = plan.sizes[g0 + g];
                    Group& d = ga.g[n_g];
                    auto half = [&](size_t at) { return reinterpret_cast<__half*>(ws + at); };
                    const float scale = i == 0 ? 1.0f / start[g0 + g] : 1.0f;  // of X, until the first apply
                    const int now = i & 1, next = now ^ 1;  // X is read from the one, A and then the new X lie in the other
                    d.rows = z.r;
                    d.count = z.count;
                    d.rest = nullptr;
                    d.rest_out = false;
                    if (mode == kGram) {
                        d.map_m = d.map_n = x_rows[g][now];
                        d.map_out = a_out[g][next];
                        d.add = nullptr;
                        d.out = half(z.x[next]);
                        d.by = scale * scale;
                        d.add_by = -shift[g];
                        d.steps = (z.k + kBK - 1) / kBK;
                    } else if (mode == kPoly) {
                        d.map_m = d.map_n = map_a[g][next];
                        d.map_out = b_out[g];
                        d.add = half(z.x[next]);
                        d.out = half(z.b);
                        d.by = poly.c;
                        d.add_by = poly.of_d(shift[g]);
                        d.steps = (z.r + kBK - 1) / kBK;
                    } else {
                        d.map_m = map_b[g];
                        d.map_out = x_out[g][next];
                        d.map_n = x_cols[g][now];
                        d.add = half(z.x[now]);
                        d.out = half(z.x[next]);
                        d.by = scale;
                        d.add_by = poly.of_x(shift[g]) * scale;
                        if (i < kRests) {
                            d.rest = ws + z.rest;
                            d.rest_by = i + 1 < kRests ? poly.a * scale : d.add_by;
                            d.rest_by *= (i == 0 ? start[g0 + g] : 1.0f) / kRestScale;
                            d.ld_rest = z.ld_rest;
                            d.rest_step = (long long)z.r * z.ld_rest;
                            d.rest_out = i + 1 < kRests;
                        }
                        d.steps = (z.r + kBK - 1) / kBK;
                    }
                    d.cols = mode == kApply ? z.k : z.r;
                    d.ld_add = d.ld_out = mode == kApply ? z.ld : z.ldr;
                    d.add_step = d.out_step = (long long)z.r * d.ld_out;
                }
                e = mode == kGram ? launch_product<kGram>(ga, pairs, s)
                                  : mode == kPoly ? launch_product<kPoly>(ga, pairs, s) : launch_product<kApply>(ga, pairs, s);
                if (e != cudaSuccess) return e;
            }
        }
    }
    if (q.iterations % 2 == 1) {
        size_t k = 0;
        for (int i = 0; i < n; ++i)
            if (plan.of[i] >= 0) {
                const Size& z = plan.sizes[plan.of[i]];
                items[k++].x = reinterpret_cast<__half*>(ws + z.x[1]) + (size_t)plan.z[i] * z.r * z.ld;
            }
    }
    return pass(items, a, true, tiles, [&](int blocks, bool vec) {
        timing_begin(kKMuonUpdate, s);
        (vec ? muon_update_kernel<true> : muon_update_kernel<false>)<<<blocks, kPassThreads, 0, s>>>(a);
        timing_end(kKMuonUpdate, s);
    });
}

}  // namespace

// (the lists are vectors: without memory for them the calls fail like one without a device)
size_t muon_workspace(const rlk_muon_matrix* t, int n) try {
    Plan p;
    plan_of(t, n, p);
    return p.bytes < 256 ? 256 : p.bytes;
} catch (const std::bad_alloc&) {
    return 0;
}

cudaError_t launch_muon(const rlk_muon_matrix* t, int n, const rlk_muon_args& q, bool step, void* workspace,
                        cudaStream_t s) try {
    return run(t, n, q, step, workspace, s);
} catch (const std::bad_alloc&) {
    return cudaErrorMemoryAllocation;
}

int read_and_clear_status_muon(cudaStream_t s) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_status_muon, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbolAsync(g_status_muon, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    return v;
}

}  // namespace rlk
