// rssm_stage_prompt.cu -- the element-wise steps of a Mamba-2 mixer block
// over packed prompts (include/rssm_stage.h): the causal conv1d + SiLU with
// the dt softplus and the conv state, the gated RMS norm, and the residual
// add with the norms around it. All are bound by the bytes they move.
#include <cmath>
#include <initializer_list>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rssm.h"
#include "rssm_stage.h"

namespace {

constexpr int kTaps = RSSM_STAGE_CONV_WIDTH;  // 4: three past inputs + the current one
constexpr int kConvThreads = 256;
constexpr int kConvTok = 16;    // tokens per CTA
constexpr int kNormThreads = 256;

__device__ __forceinline__ float bf(const __nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void set_error(int32_t* err, int32_t code) {
    if (err) atomicCAS(err, 0, code);
}

struct ConvPromptArgs {
    int batch, total, din, gn, H;
    const int32_t* cu;
    const __nv_bfloat16* zx;
    __nv_bfloat16* state;
    const float* w;
    const float* bias;
    const float* dt_bias;
    __nv_bfloat16* x;
    __nv_bfloat16* B;
    __nv_bfloat16* C;
    float* dt;
    int32_t* err;
};

// ---------------------------------------------------------------------------
// CTA (blockIdx.x, blockIdx.y): kConvTok tokens from kConvTok * blockIdx.x on,
// 256 lanes of [x | B | C | dt], one lane per thread. A thread walks its
// channel's tokens with the three inputs before the token in registers.
// The conv state of a request is read and written by one CTA alone, the one
// that holds the request's first token: it also runs the request's second
// and third token, which read the old state too, when they lie past its own
// tokens (the next CTA leaves them out), and it writes the state's new rows,
// the request's last three inputs, from the projection's rows.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kConvThreads) k_conv_prompt(const ConvPromptArgs a) {
    const int chans = a.din + 2 * a.gn;
    const size_t Dp = static_cast<size_t>(a.din) + chans + a.H;
    const int c = blockIdx.y * kConvThreads + threadIdx.x;
    const int t0 = blockIdx.x * kConvTok, t1 = min(a.total - t0, kConvTok) + t0;
    if (blockIdx.x == 0 && blockIdx.y == 0)  // every range, those without a token here too
        for (int r = threadIdx.x; r < a.batch; r += kConvThreads)
            if (a.cu[r] < 0 || a.cu[r + 1] < a.cu[r] || a.cu[r + 1] > a.total) set_error(a.err, RSSM_DEVERR_SEQ_RANGE);
    if (c >= chans + a.H) return;
    // the first request that ends past t0
    int lo = 0, hi = a.batch;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t0)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (c >= chans) {  // dt
        const int h = c - chans;
        for (int r = lo; r < a.batch; ++r) {
            const int s = a.cu[r], e = a.cu[r + 1];
            if (s >= t1) break;
            if (s < 0 || e < s || e > a.total) continue;
            for (int t = max(s, t0); t < min(e, t1); ++t) {
                const float v = bf(a.zx[t * Dp + a.din + chans + h]) + a.dt_bias[h];
                a.dt[static_cast<size_t>(t) * a.H + h] = v > 20.0f ? v : log1pf(expf(v));
            }
        }
        return;
    }
    const float4 w = reinterpret_cast<const float4*>(a.w)[c];
    const float bias = a.bias[c];
    const __nv_bfloat16* in = a.zx + a.din + c;
    __nv_bfloat16* dst;
    int width;
    if (c < a.din) {
        dst = a.x + c;
        width = a.din;
    } else if (c < a.din + a.gn) {
        dst = a.B + (c - a.din);
        width = a.gn;
    } else {
        dst = a.C + (c - a.din - a.gn);
        width = a.gn;
    }
    for (int r = lo; r < a.batch; ++r) {
        const int s = a.cu[r], e = a.cu[r + 1];
        if (s >= t1) break;
        if (s < 0 || e <= s || e > a.total) continue;
        const bool first = s >= t0;
        const int from = first ? s : max(t0, s + kTaps - 1);
        const int to = first ? max(min(e, t1), min(e, s + kTaps - 1)) : min(e, t1);
        __nv_bfloat16* st = a.state + static_cast<size_t>(r) * (kTaps - 1) * chans + c;
        __nv_bfloat16 r0, r1, r2;
        if (first) {
            r0 = st[0];
            r1 = st[chans];
            r2 = st[2 * static_cast<size_t>(chans)];
            // the last three inputs of the request, or of the old state
            const int n = e - s;
            const __nv_bfloat16 n2 = in[(e - 1) * Dp];
            const __nv_bfloat16 n1 = n >= 2 ? in[(e - 2) * Dp] : r2;
            const __nv_bfloat16 n0 = n >= 3 ? in[(e - 3) * Dp] : n == 2 ? r2 : r1;
            st[0] = n0;
            st[chans] = n1;
            st[2 * static_cast<size_t>(chans)] = n2;
        } else if (from < to) {
            r0 = in[(from - 3) * Dp];
            r1 = in[(from - 2) * Dp];
            r2 = in[(from - 1) * Dp];
        }
        for (int t = from; t < to; ++t) {
            const __nv_bfloat16 raw = in[t * Dp];
            float o = bias;
            o = fmaf(w.x, bf(r0), o);
            o = fmaf(w.y, bf(r1), o);
            o = fmaf(w.z, bf(r2), o);
            o = fmaf(w.w, bf(raw), o);
            r0 = r1;
            r1 = r2;
            r2 = raw;
            dst[static_cast<size_t>(t) * width] = __float2bfloat16_rn(o / (1.0f + expf(-o)));
        }
    }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();  // an earlier sum's readers are done
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i];
    return s;
}

// One CTA per (row, group).
__global__ void __launch_bounds__(kNormThreads) k_gate_norm_prompt(int din, int G, size_t Dp, const float* __restrict__ y,
                                                                   const __nv_bfloat16* __restrict__ zx,
                                                                   const float* __restrict__ nw, float eps,
                                                                   __nv_bfloat16* __restrict__ out) {
    __shared__ float red[kNormThreads / 32];
    const int gs = din / G;
    const size_t row = blockIdx.x;
    const size_t off = static_cast<size_t>(blockIdx.y) * gs;
    const float* yr = y + row * din + off;
    const __nv_bfloat16* zr = zx + row * Dp + off;
    auto gated = [&](int i) {
        const float z = bf(zr[i]);
        return yr[i] * (z / (1.0f + expf(-z)));
    };
    float ss = 0.f;
    for (int i = threadIdx.x; i < gs; i += kNormThreads) {
        const float g = gated(i);
        ss = fmaf(g, g, ss);
    }
    const float inv = rsqrtf(block_sum(ss, red) / static_cast<float>(gs) + eps);
    for (int i = threadIdx.x; i < gs; i += kNormThreads)
        out[row * din + off + i] = __float2bfloat16_rn(gated(i) * inv * nw[off + i]);
}

struct AddNormArgs {
    int dim;
    const void* u;
    const __nv_bfloat16* v;
    const float* post_w;
    const float* gate;
    float scale;
    const float* pre_w;
    float eps;
    void* u_out;
    __nv_bfloat16* out;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return bf(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One CTA per row.
template <typename TU>
__global__ void __launch_bounds__(kNormThreads) k_add_norm(const AddNormArgs a) {
    __shared__ float red[kNormThreads / 32];
    const size_t row = blockIdx.x;
    const int dim = a.dim;
    const TU* u = static_cast<const TU*>(a.u) + row * dim;
    TU* uo = a.u_out ? static_cast<TU*>(a.u_out) + row * dim : nullptr;
    const __nv_bfloat16* v = a.v ? a.v + row * dim : nullptr;
    float inv = 1.f;
    if (v && a.post_w) {
        float ss = 0.f;
        for (int i = threadIdx.x; i < dim; i += kNormThreads) ss = fmaf(bf(v[i]), bf(v[i]), ss);
        inv = rsqrtf(block_sum(ss, red) / static_cast<float>(dim) + a.eps);
    }
    auto stream = [&](int i) {  // u' as it is kept
        float t = to_f(u[i]);
        if (v) {
            float f = bf(v[i]);
            if (a.post_w) f = f * inv * a.post_w[i];
            if (a.gate) f *= a.gate[i];
            t = fmaf(a.scale, f, t);
        }
        TU k;
        put(&k, t);
        return k;
    };
    if (!a.out) {
        if (uo)
            for (int i = threadIdx.x; i < dim; i += kNormThreads) uo[i] = stream(i);
        return;
    }
    float ss = 0.f;
    for (int i = threadIdx.x; i < dim; i += kNormThreads) {
        const float t = to_f(stream(i));
        ss = fmaf(t, t, ss);
    }
    const float pre = rsqrtf(block_sum(ss, red) / static_cast<float>(dim) + a.eps);
    for (int i = threadIdx.x; i < dim; i += kNormThreads) {
        const TU k = stream(i);
        if (uo) uo[i] = k;
        a.out[row * dim + i] = __float2bfloat16_rn(to_f(k) * pre * a.pre_w[i]);
    }
}

rssm_status_t prompt_shape_ok(const rssm_desc_t* d) {
    if (!d) return RSSM_ERR_INVALID_ARG;
    if (d->batch < 1 || d->nheads < 1 || d->head_dim < 1 || d->d_state < 1 || d->ngroups < 1) return RSSM_ERR_SHAPE;
    if (d->nheads % d->ngroups != 0) return RSSM_ERR_SHAPE;
    const long long lanes = 2ll * d->nheads * d->head_dim + 2ll * d->ngroups * d->d_state + d->nheads;
    if (lanes > 0x7fffffffLL / 4) return RSSM_ERR_SHAPE;
    if (d->in_dtype != RSSM_BF16) return RSSM_ERR_UNSUPPORTED;
    return RSSM_OK;
}

bool aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}

rssm_status_t launched() { return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA; }

}  // namespace

extern "C" {

rssm_status_t rssm_stage_conv_prompt(const rssm_desc_t* d, int32_t total, const int32_t* cu_seqlens,
                                     const void* zxbcdt, void* conv_state, const float* conv_w, const float* conv_b,
                                     const float* dt_bias, void* x, void* B, void* C, float* dt, int32_t* err,
                                     void* stream) {
    rssm_status_t s = prompt_shape_ok(d);
    if (s != RSSM_OK) return s;
    if (total < 0 || !cu_seqlens || !conv_state || !conv_w || !conv_b || !dt_bias) return RSSM_ERR_INVALID_ARG;
    if (total == 0) return RSSM_OK;
    if (!zxbcdt || !x || !B || !C || !dt) return RSSM_ERR_INVALID_ARG;
    if (!aligned16({zxbcdt, conv_state, conv_w, conv_b, dt_bias, x, B, C, dt})) return RSSM_ERR_INVALID_ARG;
    ConvPromptArgs a;
    a.batch = d->batch;
    a.total = total;
    a.din = d->nheads * d->head_dim;
    a.gn = d->ngroups * d->d_state;
    a.H = d->nheads;
    a.cu = cu_seqlens;
    a.zx = static_cast<const __nv_bfloat16*>(zxbcdt);
    a.state = static_cast<__nv_bfloat16*>(conv_state);
    a.w = conv_w;
    a.bias = conv_b;
    a.dt_bias = dt_bias;
    a.x = static_cast<__nv_bfloat16*>(x);
    a.B = static_cast<__nv_bfloat16*>(B);
    a.C = static_cast<__nv_bfloat16*>(C);
    a.dt = dt;
    a.err = err;
    const int lanes = a.din + 2 * a.gn + a.H;
    const dim3 grid(static_cast<unsigned>((total - 1) / kConvTok + 1),
                    static_cast<unsigned>((lanes + kConvThreads - 1) / kConvThreads));
    if (grid.y > 65535) return RSSM_ERR_SHAPE;
    k_conv_prompt<<<grid, kConvThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched();
}

rssm_status_t rssm_stage_gate_norm_prompt(const rssm_desc_t* d, int32_t rows, const float* y, const void* zxbcdt,
                                          const float* norm_w, float eps, void* out, void* stream) {
    rssm_status_t s = prompt_shape_ok(d);
    if (s != RSSM_OK) return s;
    if (rows < 0 || !norm_w || !(eps > 0.0f)) return RSSM_ERR_INVALID_ARG;
    if (rows == 0) return RSSM_OK;
    if (!y || !zxbcdt || !out || !aligned16({y, zxbcdt, norm_w, out})) return RSSM_ERR_INVALID_ARG;
    const int din = d->nheads * d->head_dim, G = d->ngroups;
    const size_t Dp = 2 * static_cast<size_t>(din) + 2 * static_cast<size_t>(G) * d->d_state + d->nheads;
    if (G > 65535) return RSSM_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(G));
    k_gate_norm_prompt<<<grid, kNormThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        din, G, Dp, y, static_cast<const __nv_bfloat16*>(zxbcdt), norm_w, eps, static_cast<__nv_bfloat16*>(out));
    return launched();
}

rssm_status_t rssm_stage_add_norm(int32_t rows, int32_t dim, int32_t u_dtype, const void* u, const void* v,
                                  const float* post_w, const float* gate, float scale, const float* pre_w, float eps,
                                  void* u_out, void* out, void* stream) {
    if (rows < 0 || (u_dtype != RSSM_F32 && u_dtype != RSSM_BF16)) return RSSM_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(scale)) return RSSM_ERR_INVALID_ARG;
    if (dim < 1 || dim > 16384) return RSSM_ERR_SHAPE;
    if ((pre_w == nullptr) != (out == nullptr) && rows > 0) return RSSM_ERR_INVALID_ARG;
    if (rows == 0) return RSSM_OK;
    if (!u || (v && !u_out)) return RSSM_ERR_INVALID_ARG;
    if (!aligned16({u, v, post_w, gate, pre_w, u_out, out})) return RSSM_ERR_INVALID_ARG;
    AddNormArgs a;
    a.dim = dim;
    a.u = u;
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.post_w = post_w;
    a.gate = gate;
    a.scale = scale;
    a.pre_w = pre_w;
    a.eps = eps;
    a.u_out = u_out;
    a.out = static_cast<__nv_bfloat16*>(out);
    const unsigned grid = static_cast<unsigned>(rows);
    if (u_dtype == RSSM_F32)
        k_add_norm<float><<<grid, kNormThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    else
        k_add_norm<__nv_bfloat16><<<grid, kNormThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched();
}

}  // extern "C"
