// Rows adaln_modulation and adaln_gate_residual of RFC #386's WS1 table,
// forward and backward, for both streams of the block in one launch:
//   y = hat(x) * w * (1 + scale_b) + shift_b
//   r = x + alpha * gate_b * u,  u = h or hat(h) * w_post,  then y from r
// (the formulas and the gradients' are in include/rlk_joint_attn.h).
//
// Every kernel here is bound by HBM: a row is read once, stays in registers
// between its reductions and is written once.
#include "rlk_device.cuh"
#include "rlk_internal.h"

RLK_DEFINE_STRICT_PROBE(probe_adaln_tu)

namespace rlk {
namespace {

constexpr int kMaxThreads = 512;  // 8 columns a thread and pass: C <= 4096 in one, <= 8192 in two
constexpr int kMaxWarps = kMaxThreads / 32;

// ------------------------------------------------------------ 8 columns
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// stores 8 values and leaves in v what was stored
__device__ __forceinline__ void store8(uint16_t* p, float (&v)[8]) {
    uint4 q = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    *reinterpret_cast<uint4*>(p) = q;
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ void store8(float* p, float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// 8 values of a modulation row (or `absent` in each)
__device__ __forceinline__ void load8_mod(const void* base, bool fp32, long long at, float absent, float (&v)[8]) {
    if (base == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = absent;
    } else if (fp32) {
        load8(static_cast<const float*>(base) + at, v);
    } else {
        load8(static_cast<const uint16_t*>(base) + at, v);
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Elements of a row that warp w holds.
template <int NV>
__device__ __forceinline__ int warp_count(int w, int groups) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) n += min(max(groups - (j * (int)blockDim.x + 32 * w), 0), 32);
    return 8 * n;
}

// Mean (0 for rms) and 1 / deviation of a row held NV * 8 values a thread,
// inactive ones 0. Each warp takes its own mean and its squares about that,
// the warps are then joined about the row's mean (a large mean cancels in
// neither step), so one block barrier a row is enough. buf: kMaxWarps slots
// that the previous call must not have used.
template <int NV>
__device__ __forceinline__ float2 row_stats(const float (&v)[NV][8], const bool (&act)[NV], bool rms, int C, float eps,
                                            float2* buf) {
    const int warp = threadIdx.x / 32, n_warps = blockDim.x / 32, groups = C / 8;
    float s = 0.0f, q = 0.0f, mean_w = 0.0f;
    if (!rms) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[j][i];
        s = warp_sum(s);
        mean_w = s / (float)max(warp_count<NV>(warp, groups), 1);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (act[j])
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float z = v[j][i] - mean_w;
                q = fmaf(z, z, q);
            }
    q = warp_sum(q);
    if (threadIdx.x % 32 == 0) buf[warp] = make_float2(s, q);
    __syncthreads();
    float mean = 0.0f, m2 = 0.0f;
    if (!rms) {
        for (int w = 0; w < n_warps; ++w) mean += buf[w].x;
        mean /= (float)C;
    }
    for (int w = 0; w < n_warps; ++w) {
        const float2 p = buf[w];
        if (!rms) {
            const float n = (float)warp_count<NV>(w, groups);
            const float z = n > 0.0f ? p.x / n - mean : 0.0f;
            m2 = fmaf(n * z, z, m2);
        }
        m2 += p.y;
    }
    return make_float2(mean, 1.0f / sqrtf(m2 / (float)C + eps));
}

// Sums of two values over the block; buf as above.
__device__ __forceinline__ float2 block_sum2(float x, float y, float2* buf) {
    const int warp = threadIdx.x / 32, n_warps = blockDim.x / 32;
    x = warp_sum(x);
    y = warp_sum(y);
    if (threadIdx.x % 32 == 0) buf[warp] = make_float2(x, y);
    __syncthreads();
    float2 r = make_float2(0.0f, 0.0f);
    for (int w = 0; w < n_warps; ++w) {
        r.x += buf[w].x;
        r.y += buf[w].y;
    }
    return r;
}

// ------------------------------------------------------------ forward
// One CTA per row.
template <typename X, typename Y, int NV, bool GATE, bool POST>
__global__ void __launch_bounds__(kMaxThreads) adaln_fwd_kernel(const __grid_constant__ AdalnArgs a) {
    __shared__ float2 buf[2][kMaxWarps];
    const long long rows_txt = (long long)a.B * a.s[0].T;
    const int img = blockIdx.x >= rows_txt;
    const AdalnStream& st = a.s[img];
    const long long row = (long long)blockIdx.x - (img ? rows_txt : 0);
    const int b = (int)(row / st.T), C = a.C;
    const X* x = static_cast<const X*>(st.x) + row * C;
    float v[NV][8];
    bool act[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * blockDim.x + threadIdx.x);
        act[j] = c < C;
        if (act[j]) {
            load8(x + c, v[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        }
    }
    if (GATE) {
        float u[NV][8];
        const Y* h = static_cast<const Y*>(st.h) + row * C;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = 8 * (j * blockDim.x + threadIdx.x);
            if (act[j]) {
                load8(h + c, u[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[j][i] = 0.0f;
            }
        }
        float2 ps = make_float2(0.0f, 1.0f);
        if (POST) {
            ps = row_stats<NV>(u, act, a.post == RLK_NORM_RMS, C, a.eps, buf[1]);
            if (threadIdx.x == 0 && st.post_stats != nullptr) reinterpret_cast<float2*>(st.post_stats)[row] = ps;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = 8 * (j * blockDim.x + threadIdx.x);
            if (!act[j]) continue;
            float g[8], w[8];
            load8_mod(st.gate, a.mod_fp32, b * a.mod_stride + c, 1.0f, g);
            if (POST) load8_mod(st.w_post, true, c, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t = u[j][i];
                if (POST) t = (t - ps.x) * ps.y * w[i];
                v[j][i] = fmaf(a.alpha * g[i], t, v[j][i]);
            }
            store8(static_cast<X*>(st.r) + row * C + c, v[j]);
        }
        if (st.y == nullptr) return;
    }
    const float2 ms = row_stats<NV>(v, act, a.norm == RLK_NORM_RMS, C, a.eps, buf[0]);
    if (threadIdx.x == 0 && st.stats != nullptr) reinterpret_cast<float2*>(st.stats)[row] = ms;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * blockDim.x + threadIdx.x);
        if (!act[j]) continue;
        float w[8], sc[8], sh[8];
        load8_mod(st.w, true, c, 1.0f, w);
        load8_mod(st.scale, a.mod_fp32, b * a.mod_stride + c, 0.0f, sc);
        load8_mod(st.shift, a.mod_fp32, b * a.mod_stride + c, 0.0f, sh);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = fmaf((v[j][i] - ms.x) * ms.y, w[i] * (1.0f + sc[i]), sh[i]);
        store8(static_cast<Y*>(st.y) + row * C + c, v[j]);
    }
}

// ------------------------------------------------------------ backward
// One CTA per chunk of one (stream, sample)'s token rows, rows ascending. A
// thread owns its columns through the chunk and adds up A = sum dy * hat,
// S = sum dy and G = sum d * hat(h) (or d * h) in registers; the chunk's sums
// go to the workspace, where adaln_fold_kernel adds the chunks in order.
template <typename X, typename Y, int NV, bool GATE, bool POST>
__global__ void __launch_bounds__(kMaxThreads) adaln_bwd_kernel(const __grid_constant__ AdalnArgs a) {
    __shared__ float2 buf[4][kMaxWarps];
    const int chunks_txt = a.B * a.s[0].chunks;
    const int img = (int)blockIdx.x >= chunks_txt;
    const AdalnStream& st = a.s[img];
    const int chunk = (int)blockIdx.x - (img ? chunks_txt : 0);
    const int b = chunk / st.chunks, t0 = (chunk - b * st.chunks) * st.chunk_rows;
    const int t1 = min(t0 + st.chunk_rows, st.T), C = a.C;
    const float inv_c = 1.0f / (float)C;
    bool act[NV];
    float sum_a[NV][8], sum_s[NV][8], sum_g[NV][8], k[NV][8], kg[NV][8], wp[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * blockDim.x + threadIdx.x);
        act[j] = c < C;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_a[j][i] = sum_s[j][i] = sum_g[j][i] = k[j][i] = kg[j][i] = wp[j][i] = 0.0f;
        if (!act[j]) continue;
        float w[8], sc[8];
        load8_mod(st.w, true, c, 1.0f, w);
        load8_mod(st.scale, a.mod_fp32, b * a.mod_stride + c, 0.0f, sc);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[j][i] = w[i] * (1.0f + sc[i]);
        if (GATE) {
            load8_mod(st.gate, a.mod_fp32, b * a.mod_stride + c, 1.0f, kg[j]);
            if (POST) load8_mod(st.w_post, true, c, 1.0f, wp[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) kg[j][i] *= a.alpha;
        }
    }
    for (int t = t0; t < t1; ++t) {
        const long long row = (long long)b * st.T + t, at = row * C;
        const int par = (t & 1) * 2;
        float d[NV][8], hat[NV][8], e[NV][8];
        float rstd = 0.0f;
        if (st.dy != nullptr) {
            const float2 ms = reinterpret_cast<const float2*>(st.stats)[row];
            rstd = ms.y;
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = 8 * (j * blockDim.x + threadIdx.x);
#pragma unroll
                for (int i = 0; i < 8; ++i) hat[j][i] = e[j][i] = 0.0f;
                if (!act[j]) continue;
                load8(static_cast<const X*>(st.x) + at + c, hat[j]);
                load8(static_cast<const Y*>(st.dy) + at + c, e[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float z = (hat[j][i] - ms.x) * ms.y, dy = e[j][i];
                    sum_a[j][i] = fmaf(dy, z, sum_a[j][i]);
                    sum_s[j][i] += dy;
                    hat[j][i] = z;
                    e[j][i] = dy * k[j][i];
                    s1 += e[j][i];
                    s2 = fmaf(e[j][i], z, s2);
                }
            }
            float2 c12 = block_sum2(s1, s2, buf[par]);
            const float c1 = a.norm == RLK_NORM_RMS ? 0.0f : c12.x * inv_c, c2 = c12.y * inv_c;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] = rstd * (e[j][i] - c1 - hat[j][i] * c2);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = 8 * (j * blockDim.x + threadIdx.x);
            if (!act[j]) continue;
            if (st.dr != nullptr) {
                float dr[8];
                load8(static_cast<const X*>(st.dr) + at + c, dr);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] += dr[i];
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = d[j][i];
            store8(static_cast<X*>(st.dx) + at + c, o);
        }
        if (!GATE) continue;
        float2 ps = make_float2(0.0f, 1.0f);
        if (POST) ps = reinterpret_cast<const float2*>(st.post_stats)[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = 8 * (j * blockDim.x + threadIdx.x);
#pragma unroll
            for (int i = 0; i < 8; ++i) hat[j][i] = e[j][i] = 0.0f;
            if (!act[j]) continue;
            load8(static_cast<const Y*>(st.h) + at + c, hat[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float z = POST ? (hat[j][i] - ps.x) * ps.y : hat[j][i];
                sum_g[j][i] = fmaf(d[j][i], z, sum_g[j][i]);
                hat[j][i] = z;
                e[j][i] = d[j][i] * kg[j][i];
                if (POST) {
                    e[j][i] *= wp[j][i];
                    s1 += e[j][i];
                    s2 = fmaf(e[j][i], z, s2);
                }
            }
        }
        if (POST) {
            const float2 c12 = block_sum2(s1, s2, buf[par + 1]);
            const float c1 = a.post == RLK_NORM_RMS ? 0.0f : c12.x * inv_c, c2 = c12.y * inv_c;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) e[j][i] = ps.y * (e[j][i] - c1 - hat[j][i] * c2);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = 8 * (j * blockDim.x + threadIdx.x);
            if (act[j]) store8(static_cast<Y*>(st.dh) + at + c, e[j]);
        }
    }
    float* part = a.part + (long long)blockIdx.x * 3 * C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * blockDim.x + threadIdx.x);
        if (!act[j]) continue;
        store8(part + c, sum_a[j]);
        store8(part + C + c, sum_s[j]);
        if (GATE) store8(part + 2 * C + c, sum_g[j]);
    }
}

// Adds the chunks' column sums: 8 interleaved runs over a sample's chunks,
// each ascending, then the runs in order; weights' gradients over the samples
// ascending. blockIdx.y: (stream, which of A, S, G).
constexpr int kFoldRuns = 8;
__global__ void __launch_bounds__(32 * kFoldRuns) adaln_fold_kernel(const __grid_constant__ AdalnArgs a) {
    __shared__ float run[kFoldRuns][32];
    const int img = blockIdx.y / 3, which = blockIdx.y % 3;
    const AdalnStream& st = a.s[img];
    float* per_sample = which == 0 ? st.dscale : (which == 1 ? st.dshift : st.dgate);
    float* total = which == 0 ? st.dw : (which == 1 ? nullptr : st.dw_post);
    if (st.T == 0 || (per_sample == nullptr && total == nullptr)) return;
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane, C = a.C;
    const long long first = img ? (long long)a.B * a.s[0].chunks : 0;
    const float* w = which == 0 ? st.w : (which == 1 ? nullptr : (a.post != RLK_NORM_NONE ? st.w_post : nullptr));
    const float share = (w != nullptr && c < C ? w[c] : 1.0f) * (which == 2 ? a.alpha : 1.0f);
    float sum = 0.0f;
    for (int b = 0; b < a.B; ++b) {
        float s = 0.0f;
        if (c < C)
            for (int j = slice; j < st.chunks; j += kFoldRuns)
                s += a.part[((first + (long long)b * st.chunks + j) * 3 + which) * C + c];
        run[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && c < C) {
            s = run[0][lane];
            for (int k = 1; k < kFoldRuns; ++k) s += run[k][lane];
            if (per_sample != nullptr) per_sample[b * a.dmod_stride + c] = share * s;
            if (total != nullptr) {
                float coef = which == 0 ? 1.0f : a.alpha;
                const void* mod = which == 0 ? st.scale : st.gate;
                const long long at = b * a.mod_stride + c;
                float m = which == 0 ? 0.0f : 1.0f;
                if (mod != nullptr)
                    m = a.mod_fp32 ? static_cast<const float*>(mod)[at]
                                   : bf16_lo(static_cast<const uint16_t*>(mod)[at]);
                coef = which == 0 ? 1.0f + m : coef * m;
                sum = fmaf(coef, s, sum);
            }
        }
        __syncthreads();
    }
    if (slice == 0 && c < C && total != nullptr) total[c] = sum;
}

int threads_of(int C, int* nv) {
    const int groups = C / 8;
    *nv = groups <= kMaxThreads ? 1 : 2;
    return ((groups + *nv - 1) / *nv + 31) / 32 * 32;
}

template <typename X, typename Y, bool GATE, bool POST>
cudaError_t fwd_nv(const AdalnArgs& a, cudaStream_t s) {
    int nv;
    const int threads = threads_of(a.C, &nv);
    const long long rows = (long long)a.B * ((long long)a.s[0].T + a.s[1].T);
    if (nv == 1)
        adaln_fwd_kernel<X, Y, 1, GATE, POST><<<(unsigned)rows, threads, 0, s>>>(a);
    else
        adaln_fwd_kernel<X, Y, 2, GATE, POST><<<(unsigned)rows, threads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename X, typename Y, bool GATE, bool POST>
cudaError_t bwd_nv(const AdalnArgs& a, cudaStream_t s) {
    int nv;
    const int threads = threads_of(a.C, &nv);
    const long long chunks = (long long)a.B * (a.s[0].chunks + a.s[1].chunks);
    if (nv == 1)
        adaln_bwd_kernel<X, Y, 1, GATE, POST><<<(unsigned)chunks, threads, 0, s>>>(a);
    else
        adaln_bwd_kernel<X, Y, 2, GATE, POST><<<(unsigned)chunks, threads, 0, s>>>(a);
    return cudaGetLastError();
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

int adaln_chunk_rows(int T) { return T >= 1024 ? 16 : (T >= 128 ? 8 : 4); }

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
    bool any = false;
    for (const AdalnStream& t : a.s) any = any || t.dgate || t.dscale || t.dshift || t.dw || t.dw_post;
    if (!any) return cudaSuccess;
    timing_begin(kKAdalnFold, s);
    adaln_fold_kernel<<<dim3((a.C + 31) / 32, 6), 32 * kFoldRuns, 0, s>>>(a);
    timing_end(kKAdalnFold, s);
    return cudaGetLastError();
}

}  // namespace rlk
