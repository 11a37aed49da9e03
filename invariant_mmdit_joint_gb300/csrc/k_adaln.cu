// Rows adaln_modulation and adaln_gate_residual of RFC #386's WS1 table,
// forward and backward, for both streams of the block in one launch:
//   y = hat(x) * w * (1 + scale_b) + shift_b
//   r = x + alpha * gate_b * u,  u = h or hat(h) * w_post,  then y from r
// (the formulas and the gradients' are in include/rlk_joint_attn.h).
//
// Each activation is read once and written once: the floor is HBM (bf16, 1024^2
// guidance pair, C = 2560: 13.2 us forward, 26.3 us backward; four samples at
// 1328^2: 65 us forward with norms on both sides, 130 us backward). What it
// takes to come near it is many rows under way and few instructions: rows are
// copied ahead by cp.async, a CTA's threads keep the same columns for every
// row, and what a sample's rows share stays in registers. Measured: forward
// 18.7 us (4.8 TB/s) and 78 us (5.6 TB/s), backward with its folds 42 us (4.3
// TB/s) and 163 us (5.4 TB/s). The rest is the chain of a row's sums (about
// 1100 cycles of shuffles and one barrier), which the 20 warps that an SM's
// registers hold cover only in part, and the start and end of short launches.
#include <algorithm>

#include "rlk_device.cuh"
#include "rlk_internal.h"
#include "rlk_sm100.cuh"
RLK_DEFINE_STRICT_PROBE(probe_adaln_tu)

namespace rlk {
namespace {

using namespace sm100;

// ------------------------------------------------------------ row ring
// Rows come through a ring of shared-memory stages filled by cp.async. A
// thread copies and reads only its own 16-byte pieces, so the ring needs no
// barrier, and rows ahead are in flight without holding registers.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// ------------------------------------------------------------ 8 columns
// Eight consecutive columns of a row as four pairs of fp32 values: the packed
// instructions take half the issue slots of the scalar ones, which these
// kernels would otherwise run out of before HBM does.
struct V8 {
    uint64_t p[4];
};
__device__ __forceinline__ V8 v8_all(float x) {
    const uint64_t q = f2_pack(x, x);
    return V8{{q, q, q, q}};
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) { return f2_pack(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t pair_bf16(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return pack_bf16(lo, hi);
}
__device__ __forceinline__ V8 v8_of(uint4 q) {
    return V8{{bf16_pair(q.x), bf16_pair(q.y), bf16_pair(q.z), bf16_pair(q.w)}};
}
__device__ __forceinline__ V8 v8_of(float4 a, float4 b) {
    return V8{{f2_pack(a.x, a.y), f2_pack(a.z, a.w), f2_pack(b.x, b.y), f2_pack(b.z, b.w)}};
}
// With fp32 rows (SPLIT) a thread's eight columns are two groups of four, `half`
// apart: as one run, each 16-byte access of a warp left out every other 16
// bytes, so that a 32-byte sector went twice (fp32 modulation backward of 7 x
// 3212 rows of 1128 columns: 127 us, 91 in two groups).
template <bool SPLIT>
__device__ __forceinline__ V8 load8(const uint16_t* p, int half) {
    if (!SPLIT) return v8_of(*reinterpret_cast<const uint4*>(p));
    const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + half);
    return v8_of(make_uint4(a.x, a.y, b.x, b.y));
}
template <bool SPLIT>
__device__ __forceinline__ V8 load8(const float* p, int half) {
    return v8_of(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + (SPLIT ? half : 4)));
}
__device__ __forceinline__ float4 half_of(const V8& v, int k) {
    float4 f;
    f2_unpack(v.p[2 * k], f.x, f.y);
    f2_unpack(v.p[2 * k + 1], f.z, f.w);
    return f;
}
// Stores the values, rounded to the type, and returns what was stored.
template <bool SPLIT>
__device__ __forceinline__ V8 store8(uint16_t* p, int half, const V8& v, bool write = true) {
    const uint4 q = make_uint4(pair_bf16(v.p[0]), pair_bf16(v.p[1]), pair_bf16(v.p[2]), pair_bf16(v.p[3]));
    if (write && !SPLIT) *reinterpret_cast<uint4*>(p) = q;
    if (write && SPLIT) {
        *reinterpret_cast<uint2*>(p) = make_uint2(q.x, q.y);
        *reinterpret_cast<uint2*>(p + half) = make_uint2(q.z, q.w);
    }
    return v8_of(q);
}
template <bool SPLIT>
__device__ __forceinline__ V8 store8(float* p, int half, const V8& v, bool write = true) {
    if (write) {
        *reinterpret_cast<float4*>(p) = half_of(v, 0);
        *reinterpret_cast<float4*>(p + (SPLIT ? half : 4)) = half_of(v, 1);
    }
    return v;
}
// 8 values of a modulation row (or `absent` in each).
template <bool SPLIT>
__device__ __forceinline__ V8 load8_mod(const void* base, bool fp32, long long at, int half, float absent) {
    if (base == nullptr) return v8_all(absent);
    return fp32 ? load8<SPLIT>(static_cast<const float*>(base) + at, half)
                : load8<SPLIT>(static_cast<const uint16_t*>(base) + at, half);
}
__device__ __forceinline__ V8 operator*(const V8& a, const V8& b) {
    return V8{{mul_f2(a.p[0], b.p[0]), mul_f2(a.p[1], b.p[1]), mul_f2(a.p[2], b.p[2]), mul_f2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ V8 operator+(const V8& a, const V8& b) {
    return V8{{add_f2(a.p[0], b.p[0]), add_f2(a.p[1], b.p[1]), add_f2(a.p[2], b.p[2]), add_f2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ V8 operator-(const V8& a, const V8& b) {
    return V8{{sub_f2(a.p[0], b.p[0]), sub_f2(a.p[1], b.p[1]), sub_f2(a.p[2], b.p[2]), sub_f2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ V8 fma8(const V8& a, const V8& b, const V8& c) {
    return V8{{fma_f2(a.p[0], b.p[0], c.p[0]), fma_f2(a.p[1], b.p[1], c.p[1]), fma_f2(a.p[2], b.p[2], c.p[2]),
               fma_f2(a.p[3], b.p[3], c.p[3])}};
}
// Adds the eight values (or their products) to a pair of running sums.
__device__ __forceinline__ void sum8(uint64_t& s, const V8& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = add_f2(s, v.p[i]);
}
__device__ __forceinline__ void dot8(uint64_t& s, const V8& a, const V8& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma_f2(a.p[i], b.p[i], s);
}
__device__ __forceinline__ float pair_sum(uint64_t s) {
    float lo, hi;
    f2_unpack(s, lo, hi);
    return lo + hi;
}

// A value that the compiler keeps in a register: it would rather read special
// registers and kernel arguments anew at every use, which here cost more
// instructions a row than the sums.
template <typename T>
__device__ __forceinline__ T kept(T x) {
    asm volatile("" : "+r"(x));
    return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// The 16-byte pieces of 8 columns: one of bf16, two of fp32. Piece k of all
// threads is consecutive in a stage (PITCH = 16 bytes for each of the most
// threads the kernel is built for, so that a piece is at a fixed offset), as
// the copies want it: with a thread's own pieces together instead, each
// 16-byte copy of a warp went to another line and the 1328^2 backward took
// 229 us for 175.
template <typename T>
constexpr int kPieces = sizeof(T) / 2;
template <int PITCH, bool SPLIT>
__device__ __forceinline__ void ring_fill(uint32_t to, const uint16_t* src, int half) {
    if (SPLIT) {
        copy8(to, src);
        copy8(to + 8, src + half);
    } else {
        copy16(to, src);
    }
}
template <int PITCH, bool SPLIT>
__device__ __forceinline__ void ring_fill(uint32_t to, const float* src, int half) {
    copy16(to, src);
    copy16(to + PITCH, src + (SPLIT ? half : 4));
}
template <int PITCH>
__device__ __forceinline__ V8 ring_read(const uint8_t* at, const uint16_t*) {
    return v8_of(*reinterpret_cast<const uint4*>(at));
}
template <int PITCH>
__device__ __forceinline__ V8 ring_read(const uint8_t* at, const float*) {
    return v8_of(*reinterpret_cast<const float4*>(at), *reinterpret_cast<const float4*>(at + PITCH));
}

// ------------------------------------------------------------ sums of a row
// A CTA owns a row at a time, a thread the same NV * 8 of its columns in every
// row (the last 8 may lie past it). Sums run within a warp, then over the
// warps, both by exchanges in one order that depends on C alone.

// Sum over each half of a warp.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Values of a row that a warp holds (0 for one past the CTA's).
template <int NV>
__device__ __forceinline__ float held_by(int warp, int groups) {
    if (warp >= (int)blockDim.x / 32) return 0.0f;
    int held = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) held += min(max(groups - (j * (int)blockDim.x + 32 * warp), 0), 32);
    return 8.0f * (float)held;
}

// A thread whose last 8 columns lie past the row takes the row's last 8 once
// more, so that its loads need no branch; `last` (whether they exist) keeps
// them out of the sums and the results.
struct RowSums {
    float mine, joined;  // values of a row that this warp and warp lane % 16 hold
    float inv_mine, inv_c, inv_c_low, eps;
    bool last;
    int tid, warps;
};

// The sum over a thread's columns of what f(pair sum, j) adds up.
template <int NV, typename F>
__device__ __forceinline__ float thread_sum(bool last, F f) {
    uint64_t s = 0, e = 0;
#pragma unroll
    for (int j = 0; j + 1 < NV; ++j) f(s, j);
    f(e, NV - 1);
    const float end = last ? pair_sum(e) : 0.0f;
    return NV == 1 ? end : pair_sum(s) + end;
}

// s / C as s times 1 / C in two parts: one rounding of 1 / C alone would shift
// every row's statistics the same way. (A warp's own mean takes 1 / its columns
// rounded once: exact for a whole warp's 256 or 512, and a last bit of the mean
// for a row of one warp, C <= 256, unless C is a power of two. The backward's
// two means take the rounded 1 / C: they are small next to the row's values.)
__device__ __forceinline__ float per_column(float s, const RowSums& g) { return fmaf(s, g.inv_c, s * g.inv_c_low); }

// Mean (0 for rms) and 1 / deviation of a row. Each warp takes its own mean
// and its squares about that; the warps are then joined about the row's mean
// (a large mean cancels in neither step), so one barrier is enough. buf: 16
// slots, zero where there is no warp, that the previous call has not used.
template <int NV>
__device__ __forceinline__ float2 row_stats(const V8 (&v)[NV], bool rms, const RowSums& g, float2* buf) {
    float mean = 0.0f;
    if (!rms) mean = warp_sum(thread_sum<NV>(g.last, [&](uint64_t& s, int j) { sum8(s, v[j]); })) * g.inv_mine;
    const V8 m = v8_all(mean);
    float m2 = warp_sum(thread_sum<NV>(g.last, [&](uint64_t& s, int j) {
        const V8 z = v[j] - m;
        dot8(s, z, z);
    }));
    if (g.warps > 1) {
        if (g.tid % 32 == 0) buf[g.tid / 32] = make_float2(mean, m2);
        __syncthreads();
        const float2 p = buf[g.tid % 16];
        mean = rms ? 0.0f : per_column(half_sum(p.x * g.joined), g);
        const float z = p.x - mean;  // 0 for rms
        m2 = half_sum(fmaf(g.joined * z, z, p.y));
    }
    return make_float2(mean, 1.0f / sqrtf(per_column(m2, g) + g.eps));
}

// Sums of two values over the CTA. The halves of a warp take one value each
// (one exchange, then four steps on one value instead of five on two), and
// the warps' sums are joined the same way. buf: 16 slots for each value, zero
// as above, and 16 more for each behind them if there can be more warps.
template <bool MANY>
__device__ __forceinline__ float2 block_sum2(float x, float y, int tid, int warps, float* buf) {
    const int lane = tid % 32;
    const bool upper = lane >= 16;
    float v = half_sum((upper ? y : x) + __shfl_xor_sync(0xffffffffu, upper ? x : y, 16));
    if (warps > 1) {
        const int warp = tid / 32;
        if (lane % 16 == 0) buf[(lane & 16) + (MANY ? warp % 16 + warp / 16 * 32 : warp)] = v;
        __syncthreads();
        v = half_sum(MANY ? buf[lane] + buf[lane + 32] : buf[lane]);
    }
    const float other = __shfl_xor_sync(0xffffffffu, v, 16);
    return upper ? make_float2(other, v) : make_float2(v, other);
}

// ------------------------------------------------------------ forward
// CTA i takes the rows [i, i + 1) / grid of all. What is the same for every
// row of a sample (w * (1 + scale), shift, alpha * gate * w_post) stays in a
// thread's registers until the CTA comes to the next sample.
constexpr int kFwdStages = 3;
// CTAs of an SM that the registers are held to. A modulation's 83 a thread
// leave room for four CTAs of 160 threads; 72 and five of them are faster
// (1024^2, 19.3 -> 18.7 us). A gate with a norm after spills in more than its
// own three (78 us, 81 with four), but not with two CTAs of 256 or 320 threads,
// of which its 131 would leave one (1024^2 pair, C = 4096: 77 -> 53 us, C = 5120:
// 87 -> 63; two of 384 gained nothing, and without a norm after lost 74 -> 89).
template <int NV, int THREADS, bool GATE>
constexpr int kFwdCtas = GATE ? (THREADS == 256 || THREADS == 320 ? 2 : 1) : (THREADS >= 512 ? 1 : 820 / THREADS);

template <typename X, typename Y, int NV, int THREADS, bool GATE, bool POST>
__global__ void __launch_bounds__(THREADS, kFwdCtas<NV, THREADS, GATE>) adaln_fwd_kernel(const __grid_constant__ AdalnArgs a) {
    constexpr int PITCH = 16 * THREADS;
    constexpr int kX = NV * kPieces<X>, kRow = kX + (GATE ? NV * kPieces<Y> : 0);  // a row's pieces: x, h
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 buf[2][16];
    const int tid = kept((int)threadIdx.x), threads = blockDim.x, C = kept(a.C), warps = kept(threads / 32);
    const int col = 8 * tid;
    const bool rms = a.norm == RLK_NORM_RMS, post_rms = a.post == RLK_NORM_RMS;
    RowSums g;
    g.mine = held_by<NV>(tid / 32, C / 8);
    g.joined = held_by<NV>(tid % 16, C / 8);
    g.inv_mine = 1.0f / fmaxf(g.mine, 1.0f);
    g.inv_c = 1.0f / (float)C;
    g.inv_c_low = fmaf(-(float)C, g.inv_c, 1.0f) / (float)C;
    g.eps = a.eps;
    g.tid = tid;
    g.warps = warps;
    const bool last = g.last = 8 * (NV - 1) * threads + col < C;
    // a thread's columns: from c0 and, of NV = 2, from c0 + step
    constexpr bool S = sizeof(X) == 4;
    const int c0 = (S ? 4 : 8) * min(tid, C / 8 - 1), half = S ? C / 2 : 4;
    const int step = (S ? 4 : 8) * min(threads + tid, C / 8 - 1) - c0;
    const int rows_txt = a.B * a.s[0].T, rows = rows_txt + a.B * a.s[1].T;
    const int lo = (int)((long long)rows * blockIdx.x / gridDim.x);
    const int hi = (int)((long long)rows * (blockIdx.x + 1) / gridDim.x);
    // A bf16 residual rounds its product by itself: bf16 values times a short
    // decimal alpha are often a short number, and the sum then a tie of bf16,
    // which a single rounding of the sum misses (alpha 0.7, normal values: 157 of
    // 1.3 million on the wrong side, 524 by one fma). As an fma with -0 (eps > 0 is
    // finite): a packed product followed by a packed sum is made one fma.
    constexpr bool kTwice = GATE && !POST && sizeof(X) == 2;
    const float minus_zero = -0.0f * a.eps;
    constexpr uint32_t stage_bytes = kRow * PITCH;
    const uint32_t ring = smem_u32(smem) + 16 * tid;
    // the next row to copy: text rows of all samples, then image rows
    int fill_row = lo;
    const bool in_img = lo >= rows_txt;
    const long long at0 = (long long)(lo - (in_img ? rows_txt : 0)) * C + c0;
    const X* fx = static_cast<const X*>(a.s[in_img].x) + at0;
    const Y* fh = static_cast<const Y*>(a.s[in_img].h) + at0;
    auto fill = [&](uint32_t to) {
        if (fill_row < hi) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                ring_fill<PITCH, S>(to + PITCH * (j * kPieces<X>), fx + j * step, half);
                if (GATE) ring_fill<PITCH, S>(to + PITCH * (kX + j * kPieces<Y>), fh + j * step, half);
            }
            fx += C;
            if (GATE) fh += C;
            if (++fill_row == rows_txt) {
                fx = static_cast<const X*>(a.s[1].x) + c0;
                fh = static_cast<const Y*>(a.s[1].h) + c0;
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kFwdStages - 1; ++k) fill(ring + k * stage_bytes);
    if (tid < 32) buf[tid / 16][tid % 16] = make_float2(0.0f, 0.0f);
    __syncthreads();
    uint32_t stage = 0, filled = (kFwdStages - 1) * stage_bytes;  // to read, to fill
    int parity = 0;
    for (int row = lo; row < hi;) {
        const int img = row >= rows_txt, off = img ? rows_txt : 0;
        const AdalnStream& st = a.s[img];
        const int b = (row - off) / st.T, end = min(off + (b + 1) * st.T, hi);
        V8 k[NV], sh[NV], ga[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * step;
            const long long mod = b * a.mod_stride + c;
            k[j] = load8_mod<S>(st.w, true, c, half, 1.0f) * (v8_all(1.0f) + load8_mod<S>(st.scale, a.mod_fp32, mod, half, 0.0f));
            sh[j] = load8_mod<S>(st.shift, a.mod_fp32, mod, half, 0.0f);
            if (GATE) {
                ga[j] = v8_all(a.alpha) * load8_mod<S>(st.gate, a.mod_fp32, mod, half, 1.0f);
                if (POST) ga[j] = ga[j] * load8_mod<S>(st.w_post, true, c, half, 1.0f);
            }
        }
        const long long first = (long long)(row - off) * C + c0;
        X* rp = static_cast<X*>(st.r) + first;
        Y* yp = static_cast<Y*>(st.y) + first;
        float2* stats = reinterpret_cast<float2*>(st.stats) + (row - off);
        float2* post_stats = reinterpret_cast<float2*>(st.post_stats) + (row - off);
        const bool want_y = !GATE || st.y != nullptr;
        const bool want_stats = tid == 0 && st.stats != nullptr;
        const bool want_post = POST && tid == 0 && st.post_stats != nullptr;
        for (; row < end; ++row, rp += C, yp += C, ++stats, ++post_stats) {
            fill(ring + filled);
            filled = stage;
            copies_wait<kFwdStages - 1>();
            const uint8_t* const at = smem + 16 * tid + stage;
            stage = stage == (kFwdStages - 1) * stage_bytes ? 0 : stage + stage_bytes;
            V8 v[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = ring_read<PITCH>(at + PITCH * (j * kPieces<X>), (const X*)nullptr);
            if (GATE) {
                V8 u[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    u[j] = ring_read<PITCH>(at + PITCH * (kX + j * kPieces<Y>), (const Y*)nullptr);
                if (POST) {
                    const float2 ps = row_stats<NV>(u, post_rms, g, buf[parity]);
                    parity ^= 1;
                    if (want_post) *post_stats = ps;
                    const V8 m = v8_all(ps.x), s = v8_all(ps.y);
#pragma unroll
                    for (int j = 0; j < NV; ++j) u[j] = (u[j] - m) * s;
                }
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (kTwice) u[j] = fma8(u[j], ga[j], v8_all(minus_zero));
                    v[j] = store8<S>(rp + j * step, half, kTwice ? v[j] + u[j] : fma8(u[j], ga[j], v[j]), j + 1 < NV || last);
                }
                if (!want_y) continue;
            }
            const float2 ms = row_stats<NV>(v, rms, g, buf[parity]);
            parity ^= 1;
            if (want_stats) *stats = ms;
            const V8 m = v8_all(ms.x), s = v8_all(ms.y);
#pragma unroll
            for (int j = 0; j < NV; ++j) store8<S>(yp + j * step, half, fma8((v[j] - m) * s, k[j], sh[j]), j + 1 < NV || last);
        }
    }
    copies_wait<0>();
}

// ------------------------------------------------------------ backward
// The rows of each (stream, sample) come in chunks; CTA i takes the chunks that
// begin in the rows [i, i + 1) / grid of all. Their rows follow one another, so
// the ring runs on from chunk to chunk. A thread owns its columns and adds up A = sum
// dy * hat, S = sum dy and G = sum d * hat(h) (or d * h) in registers; a
// chunk's sums go to the workspace, where adaln_fold_kernel adds the chunks.
template <typename X, typename Y, bool GATE>
constexpr int kBwdRow = 2 * kPieces<X> + (GATE ? 2 : 1) * kPieces<Y>;  // pieces of 8 columns: x, dr, dy, h
// CTAs of an SM that the registers are held to. Without a gate 96 registers a
// thread (64 and three CTAs left the 1024^2 modulation as it was, 42 us), of
// 512 threads 64 and two CTAs (1024^2 pair at C = 4096: 64 us, 75 with one CTA
// of 101). A gate uses up to 128, and fewer CTAs that have them are faster
// (four samples at 1328^2 with a norm after: C = 768 81 -> 67 us, C = 1920 with
// 256 threads for 320 168 -> 151; the worst, 1024^2 at C = 1280 without it, 32
// -> 34), but not one of 320 threads for two, nor two of 512 of 64 registers
// (C = 4096 97 us, 125).
template <int NV, int THREADS, bool GATE>
constexpr int kBwdCtas = NV == 2 || THREADS > 512 ? 1
                         : GATE ? (THREADS == 320 ? 2 : 512 / THREADS)
                                : (THREADS == 512 ? 2 : 680 / THREADS);
// Stages: four, or as many as let that many CTAs share the shared memory.
template <typename X, typename Y, int NV, int THREADS, bool GATE>
constexpr int kBwdFit = 220 * 1024 / kBwdCtas<NV, THREADS, GATE> / (16 * THREADS * NV * kBwdRow<X, Y, GATE>);
template <typename X, typename Y, int NV, int THREADS, bool GATE>
constexpr int kBwdStages = kBwdFit<X, Y, NV, THREADS, GATE> >= 4
                               ? 4
                               : (kBwdFit<X, Y, NV, THREADS, GATE> >= 1 ? kBwdFit<X, Y, NV, THREADS, GATE> : 1);

template <typename X, typename Y, int NV, int THREADS, bool GATE, bool POST>
__global__ void __launch_bounds__(THREADS, kBwdCtas<NV, THREADS, GATE>) adaln_bwd_kernel(const __grid_constant__ AdalnArgs a) {
    constexpr int STAGES = kBwdStages<X, Y, NV, THREADS, GATE>, PITCH = 16 * THREADS;
    constexpr int kX = NV * kPieces<X>, kY = NV * kPieces<Y>;
    constexpr int kDr = kX, kDy = 2 * kX, kH = 2 * kX + kY;  // a row's pieces: x, dr, dy, h
    constexpr int kRow = 2 * kX + kY + (GATE ? kY : 0);
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr bool MANY = THREADS > 512;
    __shared__ float buf[2][MANY ? 64 : 32];
    const int tid = kept((int)threadIdx.x), threads = blockDim.x, C = kept(a.C), warps = kept(threads / 32);
    const int col = 8 * tid;
    const int units_txt = a.B * a.s[0].chunks, units = units_txt + a.B * a.s[1].chunks;
    const int rows_txt = a.B * a.s[0].T, rows = rows_txt + a.B * a.s[1].T;
    // the first chunk that begins at row i / grid of all rows or after it, and that chunk's first row
    auto share = [&](unsigned i, int& unit, int& row) {
        const int at = (int)((long long)rows * i / gridDim.x), img = at >= rows_txt, off = img ? rows_txt : 0;
        const AdalnStream& st = a.s[img];
        const int T = max(st.T, 1), b = (at - off) / T, j = (at - off - b * T + st.chunk_rows - 1) / st.chunk_rows;
        unit = (img ? units_txt : 0) + b * st.chunks + j;
        row = off + b * T + min(j * st.chunk_rows, T);
    };
    int lo, hi, row_lo, row_hi;
    share(blockIdx.x, lo, row_lo);
    share(blockIdx.x + 1, hi, row_hi);
    if (blockIdx.x + 1 == gridDim.x) hi = units, row_hi = rows;
    const float inv_c = 1.0f / (float)C;
    const bool rms = a.norm == RLK_NORM_RMS, post_rms = a.post == RLK_NORM_RMS;
    const bool last = 8 * (NV - 1) * threads + col < C;
    // a thread's columns: from c0 and, of NV = 2, from c0 + step
    constexpr bool S = sizeof(X) == 4;
    const int c0 = (S ? 4 : 8) * min(tid, C / 8 - 1), half = S ? C / 2 : 4;
    const int step = (S ? 4 : 8) * min(threads + tid, C / 8 - 1) - c0;
    constexpr uint32_t stage_bytes = kRow * PITCH;
    const uint32_t ring = smem_u32(smem) + 16 * tid;
    // the next row to copy
    int fill_row = row_lo;
    const X *fx, *fdr;
    const Y *fdy, *fh;
    // (dy and dr are given for both streams or for neither)
    const bool has_dy = a.s[row_lo >= rows_txt].dy != nullptr, has_dr = a.s[row_lo >= rows_txt].dr != nullptr;
    auto fill_from = [&](const AdalnStream& st, long long at) {
        fx = static_cast<const X*>(st.x) + at;
        fdr = static_cast<const X*>(st.dr) + at;
        fdy = static_cast<const Y*>(st.dy) + at;
        fh = static_cast<const Y*>(st.h) + at;
    };
    fill_from(a.s[row_lo >= rows_txt], (long long)(row_lo - (row_lo >= rows_txt ? rows_txt : 0)) * C + c0);
    // what is absent reads as zeros: of the ring here, of the statistics below
    if (!has_dy || !has_dr)
        for (uint32_t i = 0; i < STAGES * kRow; ++i)
            *reinterpret_cast<uint4*>(smem + 16 * tid + PITCH * i) = make_uint4(0, 0, 0, 0);
    auto fill = [&](uint32_t to) {
        if (fill_row < row_hi) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (has_dy) {
                    ring_fill<PITCH, S>(to + PITCH * (j * kPieces<X>), fx + j * step, half);
                    ring_fill<PITCH, S>(to + PITCH * (kDy + j * kPieces<Y>), fdy + j * step, half);
                }
                if (has_dr) ring_fill<PITCH, S>(to + PITCH * (kDr + j * kPieces<X>), fdr + j * step, half);
                if (GATE) ring_fill<PITCH, S>(to + PITCH * (kH + j * kPieces<Y>), fh + j * step, half);
            }
            fx += C;
            fdr += C;
            fdy += C;
            if (GATE) fh += C;
            if (++fill_row == rows_txt) fill_from(a.s[1], c0);
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fill(ring + k * stage_bytes);
    if (tid < 32)
#pragma unroll
        for (int i = 0; i < (MANY ? 64 : 32); i += 32) buf[0][i + tid] = buf[1][i + tid] = 0.0f;
    __syncthreads();
    V8 sum_a[NV], sum_s[NV], sum_g[NV], k[NV], kg[NV];
    uint32_t stage = 0, filled = (STAGES - 1) * stage_bytes;  // to read, to fill
    int parity = 0, row = row_lo, sample = -1;
    for (int unit = lo; unit < hi; ++unit) {  // (none, if the CTA's rows lie inside one chunk)
        const int img = unit >= units_txt, v = unit - (img ? units_txt : 0);
        const AdalnStream& st = a.s[img];
        const int b = v / st.chunks, t0 = (v - b * st.chunks) * st.chunk_rows;
        if (sample != img * a.B + b) {
            sample = img * a.B + b;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = c0 + j * step;
                const long long mod = b * a.mod_stride + c;
                k[j] = load8_mod<S>(st.w, true, c, half, 1.0f) * (v8_all(1.0f) + load8_mod<S>(st.scale, a.mod_fp32, mod, half, 0.0f));
                if (GATE) {
                    kg[j] = v8_all(a.alpha) * load8_mod<S>(st.gate, a.mod_fp32, mod, half, 1.0f);
                    if (POST) kg[j] = kg[j] * load8_mod<S>(st.w_post, true, c, half, 1.0f);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) sum_a[j] = sum_s[j] = sum_g[j] = v8_all(0.0f);
        const int n = min(st.chunk_rows, st.T - t0), local = row - (img ? rows_txt : 0);
        X* dx = static_cast<X*>(st.dx) + (long long)local * C + c0;
        Y* dh = static_cast<Y*>(st.dh) + (long long)local * C + c0;
        // statistics are read a row ahead
        const float2* stats = reinterpret_cast<const float2*>(st.stats) + local;
        const float2* post_stats = reinterpret_cast<const float2*>(st.post_stats) + local;
        float2 next_ms = make_float2(0.0f, 0.0f), next_ps = next_ms;
        if (has_dy) next_ms = *stats;
        if (POST) next_ps = *post_stats;
        for (int t = 0; t < n; ++t, dx += C, dh += C) {
            fill(ring + filled);
            filled = stage;
            const float2 ms = next_ms, ps = next_ps;
            if (t + 1 < n) {
                if (has_dy) next_ms = *++stats;
                if (POST) next_ps = *++post_stats;
            }
            copies_wait<STAGES - 1>();
            const uint8_t* const at = smem + 16 * tid + stage;
            stage = stage == (STAGES - 1) * stage_bytes ? 0 : stage + stage_bytes;
            V8 d[NV], hat[NV];
            {
                const V8 m = v8_all(ms.x), s = v8_all(ms.y);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const V8 dy = ring_read<PITCH>(at + PITCH * (kDy + j * kPieces<Y>), (const Y*)nullptr);
                    hat[j] = (ring_read<PITCH>(at + PITCH * (j * kPieces<X>), (const X*)nullptr) - m) * s;
                    sum_a[j] = fma8(dy, hat[j], sum_a[j]);
                    sum_s[j] = sum_s[j] + dy;
                    d[j] = dy * k[j];
                }
                const float s1 = thread_sum<NV>(last, [&](uint64_t& q, int j) { sum8(q, d[j]); });
                const float s2 = thread_sum<NV>(last, [&](uint64_t& q, int j) { dot8(q, d[j], hat[j]); });
                const float2 c12 = block_sum2<MANY>(s1, s2, tid, warps, buf[parity]);
                parity ^= 1;
                // d = dr + rstd * (e - mean(e) - hat * mean(e * hat))
                const V8 c1 = v8_all(rms ? 0.0f : -ms.y * (c12.x * inv_c)), c2 = v8_all(-ms.y * (c12.y * inv_c));
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const V8 dr = ring_read<PITCH>(at + PITCH * (kDr + j * kPieces<X>), (const X*)nullptr);
                    d[j] = dr + fma8(d[j], s, fma8(hat[j], c2, c1));
                    store8<S>(dx + j * step, half, d[j], j + 1 < NV || last);
                }
            }
            if (!GATE) continue;
            const V8 m = v8_all(ps.x), s = v8_all(ps.y);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                hat[j] = ring_read<PITCH>(at + PITCH * (kH + j * kPieces<Y>), (const Y*)nullptr);
                if (POST) hat[j] = (hat[j] - m) * s;
                sum_g[j] = fma8(d[j], hat[j], sum_g[j]);
                d[j] = d[j] * kg[j];
                if (!POST) store8<S>(dh + j * step, half, d[j], j + 1 < NV || last);
            }
            if (POST) {
                const float s1 = thread_sum<NV>(last, [&](uint64_t& q, int j) { sum8(q, d[j]); });
                const float s2 = thread_sum<NV>(last, [&](uint64_t& q, int j) { dot8(q, d[j], hat[j]); });
                const float2 c12 = block_sum2<MANY>(s1, s2, tid, warps, buf[parity]);
                parity ^= 1;
                const V8 c1 = v8_all(post_rms ? 0.0f : -ps.y * (c12.x * inv_c)), c2 = v8_all(-ps.y * (c12.y * inv_c));
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    store8<S>(dh + j * step, half, fma8(d[j], s, fma8(hat[j], c2, c1)), j + 1 < NV || last);
            }
        }
        row += n;
        float* const part = a.part + (long long)unit * 3 * C + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j + 1 == NV && !last) break;
            store8<S>(part + j * step, half, sum_a[j]);
            store8<S>(part + C + j * step, half, sum_s[j]);
            if (GATE) store8<S>(part + 2 * C + j * step, half, sum_g[j]);
        }
    }
    copies_wait<0>();
}

// Adds the chunks' column sums of one sample, stream and quantity (A, S or G;
// blockIdx.y = 3 * stream + which, z = sample): a thread takes four columns of
// every kFoldRuns-th chunk, the runs are added in order (as many as there are
// chunks, if fewer). Weights' gradients
// need every sample's sum: it replaces the sample's first chunk's, which only
// this CTA reads, for adaln_weight_kernel. 32 runs: the 256 chunks of a 4096
// token sample are eight loads a thread, all under way at once (1024^2
// modulation 42.8 -> 41.9 us with its fold, 5 samples of 1365 fp32 rows with
// the gate 42.9 -> 41.2; 64 runs of 16 columns 43.2 and 43.7).
constexpr int kFoldRuns = 32;
constexpr int kFoldColumns = 64;  // of a CTA: 16 threads
__global__ void __launch_bounds__(kFoldColumns / 4 * kFoldRuns) adaln_fold_kernel(const __grid_constant__ AdalnArgs a) {
    __shared__ float4 run[kFoldRuns][kFoldColumns / 4];
    const int img = blockIdx.y / 3, which = blockIdx.y % 3, b = blockIdx.z;
    const AdalnStream& st = a.s[img];
    float* const per_sample = which == 0 ? st.dscale : (which == 1 ? st.dshift : st.dgate);
    const float* const total = which == 0 ? st.dw : (which == 1 ? nullptr : st.dw_post);
    if (st.T == 0 || (per_sample == nullptr && total == nullptr)) return;
    const int lane = threadIdx.x % (kFoldColumns / 4), slice = threadIdx.x / (kFoldColumns / 4);
    const int c = blockIdx.x * kFoldColumns + 4 * lane, C = a.C;
    const long long first = (img ? (long long)a.B * a.s[0].chunks : 0) + (long long)b * st.chunks;
    float* const part = a.part + (first * 3 + which) * C + c;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < C)
#pragma unroll 8
        for (int j = slice; j < st.chunks; j += kFoldRuns) {
            const float4 p = *reinterpret_cast<const float4*>(part + (long long)j * 3 * C);
            s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
        }
    run[slice][lane] = s;
    const int runs = blockDim.x / (kFoldColumns / 4);
    for (int k = slice + runs; k < kFoldRuns; k += runs) run[k][lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    if (slice > 0 || c >= C) return;
#pragma unroll
    for (int k = 1; k < kFoldRuns; ++k) {
        const float4 p = run[k][lane];
        s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    if (total != nullptr) *reinterpret_cast<float4*>(part) = s;
    if (per_sample == nullptr) return;
    float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (which == 0 && st.w != nullptr) w = *reinterpret_cast<const float4*>(st.w + c);
    if (which == 2) {
        if (a.post != RLK_NORM_NONE && st.w_post != nullptr) w = *reinterpret_cast<const float4*>(st.w_post + c);
        w.x *= a.alpha, w.y *= a.alpha, w.z *= a.alpha, w.w *= a.alpha;
    }
    *reinterpret_cast<float4*>(per_sample + b * a.dmod_stride + c) =
        make_float4(w.x * s.x, w.y * s.y, w.z * s.z, w.w * s.w);
}

// dw = sum_b (1 + scale_b) * A_b and dw_post = alpha * sum_b gate_b * G_b, b
// ascending. blockIdx.y = 2 * stream + (0: dw, 1: dw_post).
__global__ void __launch_bounds__(128) adaln_weight_kernel(const __grid_constant__ AdalnArgs a) {
    const int img = blockIdx.y / 2, post = blockIdx.y % 2;
    const AdalnStream& st = a.s[img];
    float* const total = post ? st.dw_post : st.dw;
    const int c = blockIdx.x * 128 + threadIdx.x, C = a.C;
    if (st.T == 0 || total == nullptr || c >= C) return;
    const void* const mod = post ? st.gate : st.scale;
    const float* part = a.part + ((img ? (long long)a.B * a.s[0].chunks : 0) * 3 + (post ? 2 : 0)) * C + c;
    float sum = 0.0f;
#pragma unroll 4
    for (int b = 0; b < a.B; ++b) {
        const long long at = b * a.mod_stride + c;
        float m = post ? 1.0f : 0.0f;
        if (mod != nullptr)
            m = a.mod_fp32 ? static_cast<const float*>(mod)[at] : bf16_lo(static_cast<const uint16_t*>(mod)[at]);
        sum = fmaf(post ? a.alpha * m : 1.0f + m, part[(long long)b * st.chunks * 3 * C], sum);
    }
    total[c] = sum;
}

// CTAs of a kernel that the current GPU holds at once, with its dynamic
// shared memory allowed. Each kernel keeps its last answer: a program calls it
// with one width mostly, and the four kernels of a block in turn (one answer for
// all of them cost the block's calls 0.9 us of host time each).
struct Fit {
    int device = -1, threads = 0, ctas = 0;
};
cudaError_t fit(Fit& last, const void* kernel, int threads, int smem, int* ctas) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (last.device != device || last.threads != threads) {
        int sms = 0, per_sm = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        last = Fit{device, threads, sms * (per_sm > 0 ? per_sm : 1)};
    }
    *ctas = last.ctas;
    return cudaSuccess;
}

int threads_of(int C, int nv) { return ((C / 8 + nv - 1) / nv + 31) / 32 * 32; }

template <typename X, typename Y, int NV, int THREADS, bool GATE, bool POST>
cudaError_t fwd_launch(const AdalnArgs& a, cudaStream_t s) {
    constexpr int kSmem = kFwdStages * 16 * NV * (kPieces<X> + (GATE ? kPieces<Y> : 0)) * THREADS;
    const int threads = threads_of(a.C, NV);
    const auto kernel = adaln_fwd_kernel<X, Y, NV, THREADS, GATE, POST>;
    static thread_local Fit last;
    int ctas = 0;
    const cudaError_t e = fit(last, reinterpret_cast<const void*>(kernel), threads, kSmem, &ctas);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.B * ((long long)a.s[0].T + a.s[1].T);
    kernel<<<(unsigned)(rows < ctas ? rows : ctas), threads, kSmem, s>>>(a);
    return cudaGetLastError();
}
// 8 columns a thread up to C = 1024, else 16: half the warps join a row, and
// more rows are under way on an SM (1024^2 modulation 21.2 us, 25.6 with 8).
// A gate's ring of one warp is laid out for one, or it bounds the CTAs of an SM
// (8 x 3114 fp32 rows of 136 columns 18.5 us in the ring of four, 15.1).
template <typename X, typename Y, bool GATE, bool POST>
cudaError_t fwd_nv(const AdalnArgs& a, cudaStream_t s) {
    if constexpr (GATE)
        if (a.C <= 256) return fwd_launch<X, Y, 1, 32, GATE, POST>(a, s);
    if (a.C <= 1024) return fwd_launch<X, Y, 1, 128, GATE, POST>(a, s);
    if (a.C <= 2560) return fwd_launch<X, Y, 2, 160, GATE, POST>(a, s);
    if (a.C <= 4096) return fwd_launch<X, Y, 2, 256, GATE, POST>(a, s);
    if (a.C <= 5120) return fwd_launch<X, Y, 2, 320, GATE, POST>(a, s);
    if constexpr (!GATE)  // (55 -> 40 us at 6144 columns with two CTAs)
        if (a.C <= 6144) return fwd_launch<X, Y, 2, 384, GATE, POST>(a, s);
    return fwd_launch<X, Y, 2, 512, GATE, POST>(a, s);
}

template <typename X, typename Y, int NV, int THREADS, bool GATE, bool POST>
cudaError_t bwd_launch(const AdalnArgs& a, cudaStream_t s) {
    constexpr int kSmem =
        kBwdStages<X, Y, NV, THREADS, GATE> * 16 * THREADS * NV * kBwdRow<X, Y, GATE>;
    const auto kernel = adaln_bwd_kernel<X, Y, NV, THREADS, GATE, POST>;
    const int threads = threads_of(a.C, NV);
    static thread_local Fit last;
    int ctas = 0;
    const cudaError_t e = fit(last, reinterpret_cast<const void*>(kernel), threads, kSmem, &ctas);
    if (e != cudaSuccess) return e;
    const long long units = (long long)a.B * (a.s[0].chunks + a.s[1].chunks);
    kernel<<<(unsigned)(units < ctas ? units : ctas), threads, kSmem, s>>>(a);
    return cudaGetLastError();
}
// 8 columns a thread up to C = 4096, with a gate up to 6144: with 16 the sums
// and factors leave room for one CTA an SM (1024^2 modulation 47 us for 51, the
// 1328^2 gate 175 for 220), and 512 threads of 128 registers spill those of a
// gate (1024^2 pair, C = 5120: 158 us, 118 with 640 threads; C = 6144: 189 and
// 143 with 768; C = 8192 would leave 64 a thread: 232, 269 with 1024). A
// modulation at C = 6144 takes 104 us, 110 with 768. Built for these numbers
// of threads, which fix the registers' limit and the ring's layout.
template <typename X, typename Y, bool GATE, bool POST>
cudaError_t bwd_nv(const AdalnArgs& a, cudaStream_t s) {
    if (a.C <= 512) return bwd_launch<X, Y, 1, 64, GATE, POST>(a, s);
    if (a.C <= 1280) return bwd_launch<X, Y, 1, 160, GATE, POST>(a, s);
    if constexpr (GATE)
        if (a.C <= 2048) return bwd_launch<X, Y, 1, 256, GATE, POST>(a, s);
    if (a.C <= 2560) return bwd_launch<X, Y, 1, 320, GATE, POST>(a, s);
    if (a.C <= 4096) return bwd_launch<X, Y, 1, 512, GATE, POST>(a, s);
    if constexpr (GATE) {
        if (a.C <= 5120) return bwd_launch<X, Y, 1, 640, GATE, POST>(a, s);
        if (a.C <= 6144) return bwd_launch<X, Y, 1, 768, GATE, POST>(a, s);
    }
    return bwd_launch<X, Y, 2, 512, GATE, POST>(a, s);
}

template <typename X, typename Y>
cudaError_t fwd_xy(const AdalnArgs& a, bool gate, cudaStream_t s) {
    if (!gate) return fwd_nv<X, Y, false, false>(a, s);
    return a.post == RLK_NORM_NONE ? fwd_nv<X, Y, true, false>(a, s) : fwd_nv<X, Y, true, true>(a, s);
}
template <typename X, typename Y>
cudaError_t bwd_xy(const AdalnArgs& a, bool gate, cudaStream_t s) {
    if (!gate) return bwd_nv<X, Y, false, false>(a, s);
    return a.post == RLK_NORM_NONE ? bwd_nv<X, Y, true, false>(a, s) : bwd_nv<X, Y, true, true>(a, s);
}

}  // namespace

// Rows of a chunk, from T and C alone: long ones write and fold fewer sums
// (1328^2 gate, T = 6889: 160 us with 32 rows, 165 with 16, 180 with 8), short
// ones spread few rows over the SMs (1024^2 modulation, T = 4096: 49, 42, 46 us;
// T = 513: 16.3 us with 4 rows for 18.6 with 8). Narrow rows leave room for more
// CTAs, which 16-row chunks do not fill: 8 for 16 took 0.72 to 0.94 of the
// time at T = 4096 and C <= 512 and as long with 8 samples of T = 6889. At
// C = 520 .. 1280, one, two and four samples with and without a gate, it took
// 0.88 of the time in the mean at T = 4096 (0.66 to 1.10), 0.97 at 4608, 0.95 at
// 4800, 1.01 at 5200, 1.04 at 6032 (0.89 to 1.11; one sample 1.03, four 1.07) and
// 0.99 at 6889 (one sample 0.94, four 1.05). (4 rows there, and 2 below T =
// 2048, gain up to a quarter with one sample and lose as much with four.)
int adaln_chunk_rows(int T, int C) {
    if (T >= 4096) return C <= 512 || (C <= 1280 && T < 5120) ? 8 : 16;
    return T >= 2048 ? 8 : (T >= 128 ? 4 : (T > 32 ? 2 : 1));
}

cudaError_t launch_adaln_fwd(const AdalnArgs& a, bool gate, cudaStream_t s) {
    timing_begin(kKAdalnFwd, s);
    cudaError_t e;
    if (!a.x_fp32)
        e = fwd_xy<uint16_t, uint16_t>(a, gate, s);
    else
        e = a.y_fp32 ? fwd_xy<float, float>(a, gate, s) : fwd_xy<float, uint16_t>(a, gate, s);
    timing_end(kKAdalnFwd, s);
    return e;
}

cudaError_t launch_adaln_bwd(const AdalnArgs& a, bool gate, cudaStream_t s) {
    timing_begin(kKAdalnBwd, s);
    cudaError_t e;
    if (!a.x_fp32)
        e = bwd_xy<uint16_t, uint16_t>(a, gate, s);
    else
        e = a.y_fp32 ? bwd_xy<float, float>(a, gate, s) : bwd_xy<float, uint16_t>(a, gate, s);
    timing_end(kKAdalnBwd, s);
    if (e != cudaSuccess) return e;
    bool any = false, weights = false;
    for (const AdalnStream& t : a.s) {
        weights = weights || t.dw != nullptr || t.dw_post != nullptr;
        any = any || t.dgate != nullptr || t.dscale != nullptr || t.dshift != nullptr;
    }
    if (!any && !weights) return cudaSuccess;
    timing_begin(kKAdalnFold, s);
    // no more threads than chunks have use for (7 x 6 rows of 3112 columns with weights: 13.1 -> 11.1 us)
    const int runs = std::min((std::max(a.s[0].chunks, a.s[1].chunks) + 1) / 2 * 2, kFoldRuns);  // (whole warps)
    adaln_fold_kernel<<<dim3((a.C + kFoldColumns - 1) / kFoldColumns, 6, a.B), kFoldColumns / 4 * runs, 0, s>>>(a);
    e = cudaGetLastError();
    timing_end(kKAdalnFold, s);
    if (e != cudaSuccess || !weights) return e;
    timing_begin(kKAdalnWeight, s);
    adaln_weight_kernel<<<dim3((a.C + 127) / 128, 4), 128, 0, s>>>(a);
    e = cudaGetLastError();
    timing_end(kKAdalnWeight, s);
    return e;
}

}  // namespace rlk
