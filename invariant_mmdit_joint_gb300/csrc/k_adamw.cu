// The optimiser step over a list of tensors: the gradients' global norm with
// its clip factor, and AdamW with fp32 or blockwise 8-bit states (formulas and
// the states' format: include/rlk_joint_attn.h). Elementwise: the floor is HBM,
// 28 bytes an element with fp32 states (p, g, m, v read; p, m, v written), 16
// with 8-bit ones and bf16 gradients. Measured: 45 million elements, fp32
// states, 185.5 us (6.8 TB/s, the copy bandwidth); 166 million, 8-bit
// states, 455 us (5.9 TB/s, 0.86), there near the issue limit too: 83
// instructions an element (105 and 600 us with one element at a time, sqrtf
// and the division, and nothing fetched ahead).
//
// The list travels as a kernel argument (up to kMaxTensors entries), so a call
// copies nothing to the device and a captured graph holds its own list. A CTA
// takes one chunk of one tensor, found by bisection in the chunk counts. AdamW's
// chunks are as long as still gives every SM eight, 16384 elements at most (166
// million with 8-bit states took 530 us in chunks of 4096, 493 of 32768, 483
// of 16384; 34 small tensors, the largest of 39 thousand, 11.7 us in chunks of
// 16384 and 4.4 us by this rule). The norm's are always 16384, since its sums
// follow them.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "rlk_device.cuh"
#include "rlk_internal.h"
#include "rlk_sm100.cuh"

RLK_DEFINE_STRICT_PROBE(probe_adamw_tu)

namespace rlk {
namespace {

using namespace sm100;

constexpr int kMaxTensors = 256;
constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kPass = kThreads * kPerThread;  // elements a CTA covers at once
// Of an AdamW chunk; with fp32 states alone a chunk gains nothing by more than
// two (185.5 us; 186.5 with one, 196 with eight).
constexpr int kMaxPasses = 8, kMaxPasses32 = 2;
constexpr int kNormChunk = 8 * kPass;

enum : uint32_t { kGradFp32 = 1, kHasMaster = 2, kEightBit = 4 };

struct Entry {
    void* p;
    float* master;
    const void* g;
    void* m;
    void* v;
    uint8_t* ms;
    uint8_t* vs;
    long long n;
    float lr_scale, decay;
    uint32_t key, kind;
    uint32_t chunk0;  // chunks of the entries before this one
    uint32_t pad;
};
template <int N>
struct List {
    int count;
    Entry e[N];
};
// Lists of at most kFewTensors travel as a small argument (1.4 KB for 22: the
// norm and step of twelve small tensors take 9.3 us for 10.7).
constexpr int kFewTensors = 16;

template <int N>
__device__ __forceinline__ int entry_of(const List<N>& l, uint32_t chunk) {
    int lo = 0, hi = l.count;  // the last entry whose chunk0 <= chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.e[mid].chunk0 <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------ 8 elements
// Eight elements as four pairs for the packed fp32 instructions. `left`
// elements remain from p on; missing ones read as 0 and are not written.
struct V8 {
    uint64_t p[4];
};
__device__ __forceinline__ V8 pairs(const float (&v)[8]) {
    return V8{{f2_pack(v[0], v[1]), f2_pack(v[2], v[3]), f2_pack(v[4], v[5]), f2_pack(v[6], v[7])}};
}
__device__ __forceinline__ void singles(const V8& q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(q.p[i], v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ V8 all8(float x) {
    const uint64_t q = f2_pack(x, x);
    return V8{{q, q, q, q}};
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
__device__ __forceinline__ V8 load8(const float* p, int left) {
    float v[8];
    if (left >= 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
    return pairs(v);
}
__device__ __forceinline__ V8 load8(const uint16_t* p, int left) {
    float v[8];
    if (left >= 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_lo(p[i]) : 0.0f;
    }
    return pairs(v);
}
__device__ __forceinline__ void store8(float* p, int left, const V8& q) {
    float v[8];
    singles(q, v);
    if (left >= 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
    }
}
__device__ __forceinline__ void store8(uint16_t* p, int left, const V8& f) {
    float v[8];
    singles(f, v);
    const uint4 q =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    if (left >= 8) {
        *reinterpret_cast<uint4*>(p) = q;
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int left) {
    if (left >= 8) return *reinterpret_cast<const uint2*>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int left, uint2 q) {
    if (left >= 8) {
        *reinterpret_cast<uint2*>(p) = q;
    } else {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// ------------------------------------------------------------ 8-bit states
// e4m3 codes times 2^(scale - 127); scale 0 (a fresh state) reads as 0 and
// 255 as NaN, both by the multiplication itself.
__device__ __forceinline__ V8 decode8(uint2 q, uint32_t scale) {
    const uint32_t w[2] = {q.x, q.y};
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
        const float2 t = __half22float2(__half2(h));
        v.p[i] = f2_pack(t.x, t.y);
    }
    return v * all8(__uint_as_float(scale << 23));
}
// The 32-bit hash "lowbias32" of Wellons' prospector search, but for its last
// step: of x, the hash is x ^ (x >> 16), its upper half x >> 16.
__device__ __forceinline__ uint32_t hash_open(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    return x * 0x846ca68bu;
}
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
    x = hash_open(x);
    return x ^ (x >> 16);
}
// max(|a|, |b|, |c|) that keeps a NaN, and that of eight values
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float top8(const V8& q) {
    float v[8];
    singles(q, v);
    return max_abs(max_abs(v[0], v[1], v[2]), max_abs(v[3], v[4], v[5]), max_abs(v[6], v[7], 0.0f));
}
// Four threads hold a block of 32. Its scale 2^(e - 8 - 127): e is the biased
// exponent of the largest magnitude, one more where that is above 1.75 * 2^..
// so that the largest code is at most 448. Adding random bits (rnd, 16 of
// them in bits 4 .. 19 and half a unit below) under a code's last bit and
// clearing what lies under it rounds up with the remainder's share. Below the
// smallest normal code (2^-6) codes are 2^-9 apart, as the values of [2^-6,
// 2^-5) are: 2^-6 is added before and taken off after. What is left is a value
// that has a code, so that the conversion does not round again.
template <bool POSITIVE>
__device__ __forceinline__ uint2 encode8(const V8& q, float t, const uint32_t (&rnd)[8], uint32_t& scale) {
    float v[8];
    singles(q, v);
    t = max_abs(t, __shfl_xor_sync(0xffffffffu, t, 1), 0.0f);
    t = max_abs(t, __shfl_xor_sync(0xffffffffu, t, 2), 0.0f);
    const uint32_t top = __float_as_uint(t);
    const uint32_t e = max((top + 0x1fffffu) >> 23, 32u);
    const bool finite = top < 0x7f800000u;
    scale = finite ? e - 8 : 255u;
    float y[8], c[8];
    singles(q * all8(__uint_as_float((262u - e) << 23)), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fabsf(y[i]) < 0.015625f ? 0.015625f : 0.0f;
    if (!POSITIVE)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fabsf(y[i]);
    float s[8];
    singles(pairs(y) + pairs(c), s);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __uint_as_float((__float_as_uint(s[i]) + rnd[i]) & 0xfff00000u);
    singles(pairs(s) - pairs(c), s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (POSITIVE)
            s[i] = v[i] > 0.0f ? fmaxf(s[i], 0.001953125f) : s[i];
        else
            s[i] = __uint_as_float(__float_as_uint(s[i]) | (__float_as_uint(v[i]) & 0x80000000u));
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(s[2 * i], s[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint2 codes = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    return finite ? codes : make_uint2(0, 0);
}

// ------------------------------------------------------------ AdamW
struct Scalars {
    float s, b1, b2, o1, o2, inv_c2, eps, most, none, step, decay;  // step = rate / (1 - beta1^t); decay = rate * weight decay
};

// m / (sqrt(v) * c + eps), each of the two within one unit in the last place
// (the quotient of a subnormal m within two, whose residual r is below the type's
// last bit): for eight elements at once, Newton's step for the square root from the
// hardware's estimate of 1 / sqrt, and Markstein's for the quotient (q + r /
// d, r = m - d q by one fma) from its estimate of 1 / d. Written out, because
// the compiler's square root and division each carry a branch an element for
// operands that cannot occur here (they were a quarter of the 8-bit step's
// instructions). v is scaled by 2^40, so that subnormal values become normal
// ones, and kept from 0 by 2^-124, which is 2^-82 in sqrt(v): at most 2^-27 of
// eps for c <= 2^55 eps (32 for the smallest eps, 2^-50). v >= 2^86, NaN (top, the
// largest) and a c above that (the first steps with a beta2 next to 1) take sqrtf
// and the division: `most` is 2^86, or 0 for such a c.
__device__ __forceinline__ V8 quotient8(const V8& m, const V8& v, float top, float most, float c, float eps) {
    if (!(top < most)) {
        float mi[8], u[8];
        singles(m, mi);
        singles(v, u);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) u[i] = mi[i] / fmaf(sqrtf(u[i]), c, eps);
        return pairs(u);
    }
    const V8 x = fma8(v, all8(1099511627776.0f), all8(4.7019774e-38f));
    float t[8];
    singles(x, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(t[i]));
    const V8 r = pairs(t), s = x * r, ns = x * (r * all8(-1.0f));
    const V8 root = fma8(fma8(ns, s, x), r * all8(0.5f), s);
    const float c20 = c * 9.5367431640625e-7f;  // 2^-20
    const V8 d = fma8(root, all8(c20), all8(eps)), nd = fma8(root, all8(-c20), all8(-eps));
    singles(d, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t[i]));
    const V8 y = pairs(t), q = m * y;
    return fma8(fma8(nd, q, m), y, q);
}

// New m, v and p of 8 elements from g (unscaled), and the largest v (NaN if
// one is). m and v take each product and sum rounded by itself, as plain
// arithmetic does: the 8-bit codes and their blocks' scales follow from these
// bits, and one last place moves a scale in some five million. The products that
// enter the sums are fmas with -0 (k.none, not known to the compiler), since a
// packed product followed by a packed sum is made one fma otherwise.
__device__ __forceinline__ float update8(const Scalars& k, const V8& grad, V8& m, V8& v, V8& p) {
    const V8 g = grad * all8(k.s);
    const V8 none = all8(k.none);
    m = fma8(all8(k.b1), m, none) + fma8(all8(k.o1), g, none);
    v = fma8(all8(k.b2), v, none) + fma8(all8(k.o2) * g, g, none);
    const float top = top8(v);
    p = p - fma8(all8(k.decay), p, all8(k.step) * quotient8(m, v, top, k.most, k.inv_c2, k.eps));
    return top;
}
template <bool G32>
__device__ __forceinline__ V8 load_grad(const Entry& e, long long at, int left) {
    return G32 ? load8(static_cast<const float*>(e.g) + at, left) : load8(static_cast<const uint16_t*>(e.g) + at, left);
}

// One chunk with fp32 states: 28 bytes an element, and enough loads of a
// thread at once that nothing need be fetched ahead.
template <bool G32, bool MASTER>
__device__ __forceinline__ void adamw_chunk32(const Entry& e, const Scalars& k, long long i0, int passes) {
    float* const master = MASTER ? e.master : static_cast<float*>(e.p);
#pragma unroll 1
    for (int j = 0; j < passes; ++j) {
        const long long at = i0 + j * kPass + threadIdx.x * kPerThread;
        const int left = (int)min(max(e.n - at, 0LL), 8LL);
        if (left == 0) return;
        const V8 g = load_grad<G32>(e, at, left);
        V8 p = load8(master + at, left), m = load8(static_cast<const float*>(e.m) + at, left),
           v = load8(static_cast<const float*>(e.v) + at, left);
        update8(k, g, m, v, p);
        store8(master + at, left, p);
        if (MASTER) store8(static_cast<uint16_t*>(e.p) + at, left, p);
        store8(static_cast<float*>(e.m) + at, left, m);
        store8(static_cast<float*>(e.v) + at, left, v);
    }
}

// One chunk with 8-bit states. Its work an element is several times that of
// fp32 states, so the next passes' elements are copied ahead into shared
// memory meanwhile; a thread copies and reads its own bytes only, which needs
// no barrier. Piece k of all threads is consecutive in a stage.
constexpr int kRingBytes = 48 * 1024;  // four CTAs an SM
template <bool G32>
constexpr int kStageBytes = kThreads * (16 * (G32 ? 4 : 3) + 16);  // g and master in 16 bytes, the codes in 8 each
// Through L1: a thread's two 16-byte copies of its fp32 elements share sectors
// with no other thread's, and past L1 (.cg) each fetched them anew (166 million
// elements 488 us, 448 through it).
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(from) : "memory");
}
template <bool G32, bool MASTER>
__device__ __forceinline__ void adamw_chunk8(const Entry& e, const Scalars& k, long long i0, int passes, uint32_t base,
                                             uint8_t* smem) {
    constexpr int kMaster = G32 ? 2 : 1, kCodes = kMaster + 2;  // pieces before the master and the codes
    constexpr int kStep = 16 * kThreads, kStages = kRingBytes / kStageBytes<G32>;  // 3, or 2
    float* const master = MASTER ? e.master : static_cast<float*>(e.p);
    const uint8_t* const mc = static_cast<const uint8_t*>(e.m);
    const uint8_t* const vc = static_cast<const uint8_t*>(e.v);
    const uint32_t ring = smem_u32(smem);
    long long at = i0 + threadIdx.x * kPerThread;
    auto fill = [&](int j, uint32_t stage) {
        const long long i = at + (long long)j * kPass;
        if (j < passes && i + 8 <= e.n) {  // (the last elements of a tensor are loaded one by one when their turn comes)
            const uint32_t to = ring + stage + 16 * threadIdx.x;
            if (G32) {
                copy16(to, static_cast<const float*>(e.g) + i);
                copy16(to + kStep, static_cast<const float*>(e.g) + i + 4);
            } else {
                copy16(to, static_cast<const uint16_t*>(e.g) + i);
            }
            copy16(to + kMaster * kStep, master + i);
            copy16(to + (kMaster + 1) * kStep, master + i + 4);
            const uint32_t codes = ring + stage + kCodes * kStep + 8 * threadIdx.x;
            copy8(codes, mc + i);
            copy8(codes + 8 * kThreads, vc + i);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    uint32_t next_ms = 0, next_vs = 0;
    auto read_scales = [&](int j) {
        const long long i = at + (long long)j * kPass;
        if (j < passes && i < e.n) {
            next_ms = e.ms[i / 32];
            next_vs = e.vs[i / 32];
        }
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) fill(j, j * kStageBytes<G32>);
    read_scales(0);
    uint32_t stage = 0, filled = (kStages - 1) * kStageBytes<G32>;  // to read, to fill
#pragma unroll 1
    for (int j = 0; j < passes; ++j) {
        if (i0 + j * kPass >= e.n) break;  // the same for the whole CTA
        fill(j + kStages - 1, filled);
        const uint8_t* const ready = smem + stage;
        filled = stage;
        stage = stage == (kStages - 1) * kStageBytes<G32> ? 0 : stage + kStageBytes<G32>;
        uint32_t old_ms = next_ms, old_vs = next_vs;
        read_scales(j + 1);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
        const long long i = at + (long long)j * kPass;
        const int left = (int)min(max(e.n - i, 0LL), 8LL);
        V8 g, p;
        uint2 mq, vq;
        if (left == 8) {
            const uint8_t* const from = ready + 16 * threadIdx.x;
            float t[8];
            if (G32) {
                *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(from);
                *reinterpret_cast<float4*>(t + 4) = *reinterpret_cast<const float4*>(from + kStep);
                g = pairs(t);
            } else {
                g = load8(reinterpret_cast<const uint16_t*>(from), 8);
            }
            *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(from + kMaster * kStep);
            *reinterpret_cast<float4*>(t + 4) = *reinterpret_cast<const float4*>(from + (kMaster + 1) * kStep);
            p = pairs(t);
            const uint8_t* const codes = ready + kCodes * kStep + 8 * threadIdx.x;
            mq = *reinterpret_cast<const uint2*>(codes);
            vq = *reinterpret_cast<const uint2*>(codes + 8 * kThreads);
        } else {
            g = load_grad<G32>(e, i, left);
            p = load8(master + i, left);
            mq = load_codes(mc + i, left);
            vq = load_codes(vc + i, left);
            // Past the end m and v are 0, and so is their scale: the threads there take part in the exchanges of a
            // last block, which the scale kept from the pass before could turn into NaN (0 * infinity).
            if (left == 0) old_ms = old_vs = 0;
        }
        V8 m = decode8(mq, old_ms), v = decode8(vq, old_vs);
        const float top = update8(k, g, m, v, p);
        store8(master + i, left, p);
        if (MASTER) store8(static_cast<uint16_t*>(e.p) + i, left, p);
        uint32_t lo[8], hi[8];
        const uint32_t x0 = (uint32_t)i * 0x9e3779b9u + base;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            // (past the end m and v are 0)
            const uint32_t x = hash_open(x0 + (uint32_t)q * 0x9e3779b9u);
            lo[q] = ((x ^ (x >> 16)) << 4 & 0xffff0u) | 8u;
            hi[q] = (x >> 12 & 0xffff0u) | 8u;
        }
        uint32_t ms, vs;
        mq = encode8<false>(m, top8(m), lo, ms);
        vq = encode8<true>(v, top, hi, vs);
        store_codes(static_cast<uint8_t*>(e.m) + i, left, mq);
        store_codes(static_cast<uint8_t*>(e.v) + i, left, vq);
        if (threadIdx.x % 4 == 0 && left > 0) {
            e.ms[i / 32] = (uint8_t)ms;
            e.vs[i / 32] = (uint8_t)vs;
        }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

// The corrections 1 - beta1^t and 1 / sqrt(1 - beta2^t) are the same bits
// whether the host computes them from a number or the threads of a captured step
// from the device's counter: powers are products of integers (beta^(2^k) in
// units of 2^-64, cut off; relative to 1 - beta^t they are off by some 2^-64 / (1 -
// beta)), and the rest is fp32 operations that no compiler may join or split. The
// powers' table comes from the host, so that a thread multiplies as often as t
// has bits set. Captured with a counter, 45 million elements with fp32 states take
// 186 us, 184 without; 166 million with 8-bit states 465 and 453 (two fp64
// powers in every thread: 1027 and 1017).
struct Powers {
    uint64_t of[31];  // beta^(2^k) * 2^64
};
__host__ __device__ __forceinline__ uint64_t product64(uint64_t a, uint64_t b) {
#ifdef __CUDA_ARCH__
    return __umul64hi(a, b);
#else
    return (uint64_t)((unsigned __int128)a * b >> 64);
#endif
}
Powers powers_of(double beta) {
    Powers p;
    p.of[0] = (uint64_t)(beta * 0x1p64);
    for (int k = 1; k < 31; ++k) p.of[k] = product64(p.of[k - 1], p.of[k - 1]);
    return p;
}
// c1 and inv_c2 of step t in 1 .. 2^31 - 1.
__host__ __device__ __forceinline__ void corrections(const Powers& beta1, const Powers& beta2, uint32_t t, float& c1,
                                                     float& inv_c2) {
    uint64_t p1 = 0, p2 = 0;
    bool any = false;
    for (int k = 0; t != 0; ++k, t >>= 1) {
        if ((t & 1u) == 0) continue;
        p1 = any ? product64(p1, beta1.of[k]) : beta1.of[k];
        p2 = any ? product64(p2, beta2.of[k]) : beta2.of[k];
        any = true;
    }
    // 2^64 - p, which is 0 in 64 bits where p = 0
    const uint64_t e1 = 0 - p1, e2 = 0 - p2;
    c1 = p1 == 0 ? 1.0f : (float)e1 * 0x1p-64f;
    // 1 / sqrt(c) by a Newton step about the fp32 root, with c and the root's square in two parts each
    float c = (float)e2, low = 0.0f;
    if (p2 == 0)
        c = 0x1p64f;
    else
        low = c == 0x1p64f ? -(float)p2 : (float)(int64_t)(e2 - (uint64_t)c);
    c *= 0x1p-64f;
    low *= 0x1p-64f;
    const float y = 1.0f / sqrtf(c), s = y * y;
    inv_c2 = fmaf(0.5f * y, fmaf(-low, s, fmaf(-c, fmaf(y, y, -s), fmaf(-c, s, 1.0f))), y);
}

struct StepArgs {
    double lr;
    float b1, b2, o1, o2, eps;
    float c1, inv_c2;      // 1 - beta1^t and 1 / sqrt(1 - beta2^t),
    Powers beta1, beta2;   // or what they follow from if step_dev
    const float* lr_dev;
    const long long* step_dev;
    const float* grad_scale;
    uint32_t seed, step;
    int passes;  // of a chunk
};

// ANY8: whether some tensor of the list has 8-bit states. fp32 ones alone take
// three CTAs an SM: with the registers of four the compiler no longer has all
// loads of a thread under way at once (45 million elements 185.5 us, 204).
template <int N, bool ANY8>
__global__ void __launch_bounds__(kThreads, ANY8 ? 4 : 3) adamw_kernel(const __grid_constant__ List<N> l,
                                                            const __grid_constant__ StepArgs a) {
    Scalars k;
    k.s = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    if (!isfinite(k.s)) return;
    const Entry& e = l.e[entry_of(l, blockIdx.x)];
    float c1 = a.c1;
    k.inv_c2 = a.inv_c2;
    uint32_t step = a.step;
    if (a.step_dev != nullptr) {
        const long long t = *a.step_dev;
        if (t < 1 || t > 0x7fffffffLL) return;  // 1 - beta^0 would make every element infinite or NaN
        step = (uint32_t)t;
        corrections(a.beta1, a.beta2, step, c1, k.inv_c2);
    }
    const double lr = a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr;
    const float rate = (float)lr * e.lr_scale;
    k.b1 = a.b1;
    k.b2 = a.b2;
    k.o1 = a.o1;
    k.o2 = a.o2;
    k.eps = a.eps;
    k.most = k.inv_c2 <= 0x1p55f * a.eps ? 0x1p86f : 0.0f;
    k.none = -0.0f * a.eps;
    k.step = rate / c1;
    k.decay = rate * e.decay;
    const long long i0 = (long long)(blockIdx.x - e.chunk0) * a.passes * kPass;
    extern __shared__ __align__(16) uint8_t smem[];  // the ring of 8-bit states
    switch (ANY8 ? e.kind : e.kind & ~kEightBit) {
        case 0: adamw_chunk32<false, false>(e, k, i0, a.passes); break;
        case kGradFp32: adamw_chunk32<true, false>(e, k, i0, a.passes); break;
        case kHasMaster: adamw_chunk32<false, true>(e, k, i0, a.passes); break;
        case kHasMaster | kGradFp32: adamw_chunk32<true, true>(e, k, i0, a.passes); break;
        default:
            if (ANY8) {
                const uint32_t base = hash32(hash32(hash32(a.seed) ^ step) ^ e.key);
                switch (e.kind & ~kEightBit) {
                    case 0: adamw_chunk8<false, false>(e, k, i0, a.passes, base, smem); break;
                    case kGradFp32: adamw_chunk8<true, false>(e, k, i0, a.passes, base, smem); break;
                    case kHasMaster: adamw_chunk8<false, true>(e, k, i0, a.passes, base, smem); break;
                    default: adamw_chunk8<true, true>(e, k, i0, a.passes, base, smem); break;
                }
            }
    }
}

// ------------------------------------------------------------ gradient norm
// A chunk's squares: a thread's in order, then its warp's by exchanges, then
// the eight warps ascending, in fp32: 76 roundings in a row at most, 2^-18 of
// the chunk's sum and half that of the norm (a few 2^-24 as roundings fall), and
// the range that the header states. An SM does two fp64 fmas a cycle: 45 million
// squares in fp64 would take 70 us. 45 million bf16 gradients are 90 MB, 13 us at the
// copy bandwidth; norm, fold and the step that follows take 207 us, 22 of them
// for the first two (26 with a check of the bounds at each load).
template <bool G32>
__device__ __forceinline__ float thread_squares(const Entry& e, long long i0, int tid) {
    float s = 0.0f;
    auto add = [&](const V8& v) {
        float g[8];
        singles(v, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(g[i], g[i], s);
    };
    constexpr int kPasses = kNormChunk / kPass;
    const long long at = i0 + tid * kPerThread;
    if (e.n - i0 >= kNormChunk) {  // no bounds to look at between the loads
        V8 v[kPasses];
#pragma unroll
        for (int j = 0; j < kPasses; ++j) v[j] = load_grad<G32>(e, at + j * kPass, 8);
#pragma unroll
        for (int j = 0; j < kPasses; ++j) add(v[j]);
    } else {
#pragma unroll 1
        for (int j = 0; j < kPasses; ++j) add(load_grad<G32>(e, at + j * kPass, (int)min(max(e.n - at - j * kPass, 0LL), 8LL)));
    }
    return s;
}
template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ List<N> l, float* part) {
    __shared__ float sums[kThreads / 32];
    const Entry& e = l.e[entry_of(l, blockIdx.x)];
    const long long i0 = (long long)(blockIdx.x - e.chunk0) * kNormChunk;
    float s = (e.kind & kGradFp32) ? thread_squares<true>(e, i0, threadIdx.x) : thread_squares<false>(e, i0, threadIdx.x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = sums[0];
        for (int w = 1; w < kThreads / 32; ++w) sum += sums[w];
        part[blockIdx.x] = sum;
    }
}

// The list's sum from its chunks', and what follows from it. One CTA, bound by
// latency: only the sum over the list is in fp64, which is what grows long. Its
// root in fp32 is two roundings more of a value that the chunks leave some units
// off anyway (in fp64, and with 32 warps' sums added one by one, 1 us longer).
__global__ void __launch_bounds__(1024) grad_norm_fold_kernel(const float* part, long long n, float pre, float max_norm,
                                                              float* out) {
    __shared__ double ws[32];
    double s = 0.0;
#pragma unroll 8
    for (long long i = threadIdx.x; i < n; i += 1024) s += (double)part[i];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (threadIdx.x % 32 == 0) ws[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    s = ws[threadIdx.x];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (threadIdx.x == 0) {
        const float norm = pre * sqrtf((float)s);
        out[0] = norm;
        float f = pre;
        if (max_norm < norm + 1e-6f) f = pre * (max_norm / (norm + 1e-6f));
        out[1] = isfinite(norm) ? f : __int_as_float(0x7fc00000);
    }
}

// ------------------------------------------------------------ lists
long long chunks_of(long long n, int chunk) { return (n + chunk - 1) / chunk; }

// Calls f(list, first chunk, chunks) for runs of at most kMaxTensors tensors
// and 2^30 chunks (a tensor's chunks stay together: n <= 2^40 elements are
// at most 2^28 chunks).
template <typename F>
cudaError_t for_lists(const rlk_adamw_tensor* t, int n, int chunk, F f) {
    constexpr long long kMaxChunks = 1LL << 30;
    List<kMaxTensors> l;
    l.count = 0;
    long long chunks = 0, first = 0;
    for (int i = 0; i <= n; ++i) {
        const long long c = i < n ? chunks_of(t[i].n, chunk) : 0;
        if (i == n || l.count == kMaxTensors || chunks + c > kMaxChunks) {
            if (l.count > 0) {
                const cudaError_t e = f(l, first, chunks);
                if (e != cudaSuccess) return e;
            }
            first += chunks;
            l.count = 0;
            chunks = 0;
        }
        if (i == n || t[i].n == 0) continue;
        Entry& d = l.e[l.count++];
        d.p = t[i].p;
        d.master = t[i].master;
        d.g = t[i].g;
        d.m = t[i].m;
        d.v = t[i].v;
        d.ms = t[i].m_scale;
        d.vs = t[i].v_scale;
        d.n = t[i].n;
        d.lr_scale = (float)t[i].lr_scale;
        d.decay = (float)t[i].weight_decay;
        d.key = t[i].key;
        d.kind = (t[i].g_dtype == RLK_FP32 ? kGradFp32 : 0u) | (t[i].master != nullptr ? kHasMaster : 0u) |
                 (t[i].state_bits == 8 ? kEightBit : 0u);
        d.chunk0 = (uint32_t)chunks;
        d.pad = 0;
        chunks += c;
    }
    return cudaSuccess;
}
List<kFewTensors> few(const List<kMaxTensors>& l) {
    List<kFewTensors> s;
    s.count = l.count;
    std::copy(l.e, l.e + l.count, s.e);
    return s;
}

}  // namespace

size_t grad_norm_partials(const rlk_adamw_tensor* t, int n) {
    size_t c = 0;
    for (int i = 0; i < n; ++i) c += (size_t)chunks_of(t[i].n, kNormChunk);
    return c;
}

cudaError_t launch_grad_norm(const rlk_adamw_tensor* t, int n, float pre, float max_norm, float* out, float* part,
                             cudaStream_t s) {
    const cudaError_t e = for_lists(t, n, kNormChunk, [&](const List<kMaxTensors>& l, long long first, long long chunks) {
        timing_begin(kKGradNorm, s);
        if (l.count <= kFewTensors)
            grad_norm_kernel<<<(unsigned)chunks, kThreads, 0, s>>>(few(l), part + first);
        else
            grad_norm_kernel<<<(unsigned)chunks, kThreads, 0, s>>>(l, part + first);
        timing_end(kKGradNorm, s);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    timing_begin(kKGradNormFold, s);
    grad_norm_fold_kernel<<<1, 1024, 0, s>>>(part, (long long)grad_norm_partials(t, n), pre, max_norm, out);
    timing_end(kKGradNormFold, s);
    return cudaGetLastError();
}

cudaError_t launch_adamw(const rlk_adamw_tensor* t, int n, const rlk_adamw_args& r, cudaStream_t s) {
    StepArgs a;
    a.lr = r.lr;
    a.b1 = (float)r.beta1;
    a.b2 = (float)r.beta2;
    a.o1 = (float)(1.0 - r.beta1);
    a.o2 = (float)(1.0 - r.beta2);
    a.eps = (float)r.eps;
    a.beta1 = powers_of(r.beta1);
    a.beta2 = powers_of(r.beta2);
    a.c1 = a.inv_c2 = 1.0f;
    if (r.step_dev == nullptr) corrections(a.beta1, a.beta2, (uint32_t)r.step, a.c1, a.inv_c2);
    a.lr_dev = r.lr_dev;
    a.step_dev = reinterpret_cast<const long long*>(r.step_dev);
    a.grad_scale = r.grad_scale;
    a.seed = r.seed;
    a.step = (uint32_t)r.step;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // (elementwise: the chunks change no byte)
    bool any8 = false;
    for (int i = 0; i < n; ++i) any8 = any8 || t[i].state_bits == 8;
    for (a.passes = any8 ? kMaxPasses : kMaxPasses32; a.passes > 1; a.passes /= 2) {
        long long chunks = 0;
        for (int i = 0; i < n; ++i) chunks += chunks_of(t[i].n, a.passes * kPass);
        if (chunks >= 8LL * sms) break;
    }
    return for_lists(t, n, a.passes * kPass, [&](const List<kMaxTensors>& l, long long, long long chunks) {
        int smem = 0;
        for (int i = 0; i < l.count; ++i)
            if (l.e[i].kind & kEightBit)
                smem = kRingBytes;
        auto launch = [&](auto kernel, const auto& list) {
            kernel<<<(unsigned)chunks, kThreads, smem, s>>>(list, a);
        };
        timing_begin(kKAdamw, s);
        if (l.count <= kFewTensors)
            smem > 0 ? launch(adamw_kernel<kFewTensors, true>, few(l)) : launch(adamw_kernel<kFewTensors, false>, few(l));
        else
            smem > 0 ? launch(adamw_kernel<kMaxTensors, true>, l) : launch(adamw_kernel<kMaxTensors, false>, l);
        timing_end(kKAdamw, s);
        return cudaGetLastError();
    });
}

}  // namespace rlk
