// The optimiser step over a list of tensors: the gradients' global norm with
// its clip factor, and AdamW with fp32 or blockwise 8-bit states (formulas and
// the states' format: include/rlk_joint_attn.h). Elementwise and bound by HBM:
// 28 bytes an element with fp32 states (p, g, m, v read; p, m, v written), 16
// with 8-bit ones and bf16 gradients.
//
// The list travels as a kernel argument (up to kMaxTensors entries), so a call
// copies nothing to the device and a captured graph holds its own list. A CTA
// takes one chunk of one tensor, found by bisection in the chunk counts.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "rlk_device.cuh"
#include "rlk_internal.h"

RLK_DEFINE_STRICT_PROBE(probe_adamw_tu)

namespace rlk {
namespace {

constexpr int kMaxTensors = 256;
constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kPass = kThreads * kPerThread;  // elements a CTA covers at once
constexpr int kChunk = 2 * kPass;

enum : uint32_t { kGradFp32 = 1, kMaster = 2, kEightBit = 4 };

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
struct List {
    int count;
    Entry e[kMaxTensors];
};

__device__ __forceinline__ int entry_of(const List& l, uint32_t chunk) {
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
// `left` elements remain from p on; missing ones read as 0 and are not written.
__device__ __forceinline__ void load8(const float* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_lo(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void store8(float* p, int left, const float (&v)[8]) {
    if (left >= 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
    }
}
__device__ __forceinline__ void store8(uint16_t* p, int left, const float (&v)[8]) {
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
__device__ __forceinline__ void decode8(uint2 q, uint8_t scale, float (&v)[8]) {
    const float f = __uint_as_float((uint32_t)scale << 23);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
        const float2 t = __half22float2(__half2(h));
        v[2 * i] = t.x * f;
        v[2 * i + 1] = t.y * f;
    }
}
// The 32-bit hash with the least bias of Wellons' prospector search.
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ (x >> 16);
}
// Four threads hold a block of 32. Its scale 2^(e - 8 - 127): e is the biased
// exponent of the largest magnitude, one more where that is above 1.75 * 2^..
// so that the largest code is at most 448. Below the smallest normal code
// (2^-6) codes are 2^-9 apart, as the values of [2^-6, 2^-5) are: adding 2^-6
// puts both ranges under one integer rounding. Adding the random bits below
// the code's last bit and truncating rounds up with the remainder's share.
template <bool POSITIVE>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], const uint32_t (&rnd)[8], uint8_t& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (top >= 0x7f800000u) {
        scale = 255;
        return make_uint2(0, 0);
    }
    const uint32_t e = max((top + 0x1fffffu) >> 23, 32u);
    scale = (uint8_t)(e - 8);
    const float f = __uint_as_float((262u - e) << 23);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = fabsf(v[i]) * f;
        const bool small = y < 0.015625f;
        const uint32_t bits = __float_as_uint(small ? y + 0.015625f : y);
        uint32_t code = ((bits + ((rnd[i] << 4) | 8u)) >> 20) - (small ? 968u : 960u);
        if (POSITIVE) {
            if (v[i] > 0.0f) code = max(code, 1u);
        } else {
            code |= (__float_as_uint(v[i]) >> 24) & 0x80u;
        }
        w[i / 4] |= code << (8 * (i % 4));
    }
    return make_uint2(w[0], w[1]);
}

// ------------------------------------------------------------ AdamW
struct Scalars {
    float s, b1, b2, o1, o2, inv_c2, eps, step, decay;  // step = rate / (1 - beta1^t); decay = rate * weight decay
};

template <bool G32, bool MASTER, bool Q8>
__device__ __forceinline__ void adamw_chunk(const Entry& e, const Scalars& k, long long i0, uint32_t base) {
#pragma unroll 1
    for (int j = 0; j < kChunk / kPass; ++j) {
        const long long at = i0 + j * kPass + threadIdx.x * kPerThread;
        if (i0 + j * kPass >= e.n) return;  // the same for the whole CTA
        const int left = (int)min(max(e.n - at, 0LL), 8LL);
        float g[8], p[8], m[8], v[8];
        float* const master = MASTER ? e.master : static_cast<float*>(e.p);
        if (G32)
            load8(static_cast<const float*>(e.g) + at, left, g);
        else
            load8(static_cast<const uint16_t*>(e.g) + at, left, g);
        load8(master + at, left, p);
        if (Q8) {
            const uint2 mq = load_codes(static_cast<const uint8_t*>(e.m) + at, left);
            const uint2 vq = load_codes(static_cast<const uint8_t*>(e.v) + at, left);
            decode8(mq, left > 0 ? e.ms[at / 32] : 0, m);
            decode8(vq, left > 0 ? e.vs[at / 32] : 0, v);
        } else {
            load8(static_cast<const float*>(e.m) + at, left, m);
            load8(static_cast<const float*>(e.v) + at, left, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gs = __fmul_rn(g[i], k.s);
            m[i] = __fadd_rn(__fmul_rn(k.b1, m[i]), __fmul_rn(k.o1, gs));
            v[i] = __fadd_rn(__fmul_rn(k.b2, v[i]), __fmul_rn(__fmul_rn(k.o2, gs), gs));
            const float u = m[i] / fmaf(sqrtf(v[i]), k.inv_c2, k.eps);
            p[i] -= fmaf(k.decay, p[i], k.step * u);
        }
        store8(master + at, left, p);
        if (MASTER) store8(static_cast<uint16_t*>(e.p) + at, left, p);
        if (Q8) {
            uint32_t lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = hash32((uint32_t)(at + i) * 0x9e3779b9u + base);
                lo[i] = r & 0xffffu;
                hi[i] = r >> 16;
            }  // (past the end m and v are 0)
            uint8_t ms, vs;
            const uint2 mq = encode8<false>(m, lo, ms), vq = encode8<true>(v, hi, vs);
            store_codes(static_cast<uint8_t*>(e.m) + at, left, mq);
            store_codes(static_cast<uint8_t*>(e.v) + at, left, vq);
            if (threadIdx.x % 4 == 0 && left > 0) {
                e.ms[at / 32] = ms;
                e.vs[at / 32] = vs;
            }
        } else {
            store8(static_cast<float*>(e.m) + at, left, m);
            store8(static_cast<float*>(e.v) + at, left, v);
        }
    }
}

struct StepArgs {
    double lr, b1, b2;
    float o1, o2, eps;
    float c1, inv_c2;  // 1 - beta1^t and 1 / sqrt(1 - beta2^t), unless step_dev
    const float* lr_dev;
    const long long* step_dev;
    const float* grad_scale;
    uint32_t seed, step;
};

__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ List l,
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
        step = (uint32_t)t;
        c1 = (float)(1.0 - pow(a.b1, (double)t));
        k.inv_c2 = (float)(1.0 / sqrt(1.0 - pow(a.b2, (double)t)));
    }
    const double lr = a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr;
    const float rate = (float)lr * e.lr_scale;
    k.b1 = (float)a.b1;
    k.b2 = (float)a.b2;
    k.o1 = a.o1;
    k.o2 = a.o2;
    k.eps = a.eps;
    k.step = rate / c1;
    k.decay = rate * e.decay;
    const long long i0 = (long long)(blockIdx.x - e.chunk0) * kChunk;
    const uint32_t base = hash32(hash32(hash32(a.seed) ^ step) ^ e.key);
    switch (e.kind) {
        case 0: adamw_chunk<false, false, false>(e, k, i0, base); break;
        case kGradFp32: adamw_chunk<true, false, false>(e, k, i0, base); break;
        case kMaster: adamw_chunk<false, true, false>(e, k, i0, base); break;
        case kMaster | kGradFp32: adamw_chunk<true, true, false>(e, k, i0, base); break;
        case kEightBit: adamw_chunk<false, false, true>(e, k, i0, base); break;
        case kEightBit | kGradFp32: adamw_chunk<true, false, true>(e, k, i0, base); break;
        case kEightBit | kMaster: adamw_chunk<false, true, true>(e, k, i0, base); break;
        default: adamw_chunk<true, true, true>(e, k, i0, base); break;
    }
}

// ------------------------------------------------------------ gradient norm
// One partial per chunk: a thread's squares in order, then a fixed tree.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ List l, float* part) {
    __shared__ float ws[kThreads / 32];
    const Entry& e = l.e[entry_of(l, blockIdx.x)];
    const long long i0 = (long long)(blockIdx.x - e.chunk0) * kChunk;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kChunk / kPass; ++j) {
        const long long at = i0 + j * kPass + threadIdx.x * kPerThread;
        const int left = (int)min(max(e.n - at, 0LL), 8LL);
        float g[8];
        if (e.kind & kGradFp32)
            load8(static_cast<const float*>(e.g) + at, left, g);
        else
            load8(static_cast<const uint16_t*>(e.g) + at, left, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(g[i], g[i], s);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (threadIdx.x % 32 == 0) ws[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) s += ws[w];
        part[blockIdx.x] = s;
    }
}

__global__ void __launch_bounds__(1024) grad_norm_fold_kernel(const float* part, long long n, float pre, float max_norm,
                                                              float* out) {
    __shared__ double ws[32];
    double s = 0.0;
    for (long long i = threadIdx.x; i < n; i += 1024) s += (double)part[i];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (threadIdx.x % 32 == 0) ws[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) s += ws[w];
        const float norm = (float)((double)pre * sqrt(s));
        out[0] = norm;
        float f = pre;
        if (max_norm < norm + 1e-6f) f = pre * (max_norm / (norm + 1e-6f));
        out[1] = isfinite(norm) ? f : __int_as_float(0x7fc00000);
    }
}

long long chunks_of(long long n) { return (n + kChunk - 1) / kChunk; }

// Calls f(list, first chunk, chunks) for runs of at most kMaxTensors tensors
// and max_chunks chunks (a tensor's chunks stay together: n <= 2^40 elements
// are 2^28 chunks).
template <typename F>
cudaError_t for_lists(const rlk_adamw_tensor* t, int n, F f) {
    constexpr long long kMaxChunks = 1LL << 30;
    List l;
    l.count = 0;
    long long chunks = 0, first = 0;
    for (int i = 0; i <= n; ++i) {
        const long long c = i < n ? chunks_of(t[i].n) : 0;
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
        d.kind = (t[i].g_dtype == RLK_FP32 ? kGradFp32 : 0u) | (t[i].master != nullptr ? kMaster : 0u) |
                 (t[i].state_bits == 8 ? kEightBit : 0u);
        d.chunk0 = (uint32_t)chunks;
        d.pad = 0;
        chunks += c;
    }
    return cudaSuccess;
}

}  // namespace

size_t grad_norm_partials(const rlk_adamw_tensor* t, int n) {
    size_t c = 0;
    for (int i = 0; i < n; ++i) c += (size_t)chunks_of(t[i].n);
    return c;
}

cudaError_t launch_grad_norm(const rlk_adamw_tensor* t, int n, float pre, float max_norm, float* out, float* part,
                             cudaStream_t s) {
    const cudaError_t e = for_lists(t, n, [&](const List& l, long long first, long long chunks) {
        timing_begin(kKGradNorm, s);
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
    a.b1 = r.beta1;
    a.b2 = r.beta2;
    a.o1 = (float)(1.0 - r.beta1);
    a.o2 = (float)(1.0 - r.beta2);
    a.eps = (float)r.eps;
    a.c1 = (float)(1.0 - std::pow(r.beta1, (double)r.step));
    a.inv_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(r.beta2, (double)r.step)));
    a.lr_dev = r.lr_dev;
    a.step_dev = reinterpret_cast<const long long*>(r.step_dev);
    a.grad_scale = r.grad_scale;
    a.seed = r.seed;
    a.step = (uint32_t)r.step;
    return for_lists(t, n, [&](const List& l, long long, long long chunks) {
        timing_begin(kKAdamw, s);
        adamw_kernel<<<(unsigned)chunks, kThreads, 0, s>>>(l, a);
        timing_end(kKAdamw, s);
        return cudaGetLastError();
    });
}

}  // namespace rlk
