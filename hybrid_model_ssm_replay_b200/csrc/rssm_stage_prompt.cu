// rssm_stage_prompt.cu -- the element-wise steps of a Mamba-2 mixer block
// over packed prompts (include/rssm_stage.h): the causal conv1d + SiLU with
// the dt softplus and the conv state, the gated RMS norm, and the residual
// add with the norms around it. All are bound by the bytes they move.
#include <atomic>
#include <cmath>
#include <initializer_list>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rssm.h"
#include "rssm_internal.h"
#include "rssm_stage.h"

namespace {

constexpr int kTaps = RSSM_STAGE_CONV_WIDTH;  // 4: three past inputs + the current one
constexpr int kConvThreads = 256;
constexpr int kNormThreads = 256;

__device__ __forceinline__ float bf(const __nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void set_error(int32_t* err, int32_t code) {
    if (err) atomicCAS(err, 0, code);
}

struct ConvPromptArgs {
    int batch, total, din, gn, H;
    int tok;     // tokens per CTA
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

// silu as rssm_stage_conv forms it, in bf16.
__device__ __forceinline__ uint16_t silu_exact(float o) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(o / (1.0f + expf(-o))));
}

// Two fp32 lanes in one instruction, each as the scalar one rounds.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// silu of two channels as a pair of bf16, the bits of silu_exact for less:
// o / (1 + 2^(-o log2 e)) with the approximate exponential and one
// approximate reciprocal r of both denominators' product, 1/a = b r. For
// o > -32 that is within 26 fp32 spacings of the quotient (19 from the
// argument -o log2 e, up to 46 in size, 2 of ex2, 1 of rcp, 4 of the add and
// the products) and the library form within 3. So when 1 - 2^-18 and 1 + 2^-18
// times it round to the same bf16, the library form does too; else (one value
// in a thousand), and when r is NaN or so small that an o may be below -32,
// the library form decides.
__device__ __forceinline__ uint32_t silu2(float2 o) {
    const float2 t = mul2(o, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.0f, 1.0f));
    const float r = rcp_approx(d.x * d.y);
    const float2 v = mul2(o, mul2(make_float2(d.y, d.x), make_float2(r, r)));
    constexpr float kUp = 1.0f + 1.0f / 262144.0f, kDown = 1.0f - 1.0f / 262144.0f;
    const float2 lo = mul2(v, make_float2(kDown, kDown)), hi = mul2(v, make_float2(kUp, kUp));
    uint32_t w = pack_bf16(lo.x, lo.y);
    if (!(r > 1.4210854715202004e-14f) || w != pack_bf16(hi.x, hi.y))  // 2^-46
        w = silu_exact(o.x) | (static_cast<uint32_t>(silu_exact(o.y)) << 16);
    return w;
}

// The first request that ends past token t: each lane tries a part of the range.
__device__ __forceinline__ int first_request(const int32_t* cu, int batch, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = batch;
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5, r = lo + lane * step;
        const unsigned past = __ballot_sync(0xffffffffu, r < hi && cu[r + 1] <= t);
        const int n = __popc(past);
        if (n == 0) break;
        hi = min(hi, lo + n * step);
        lo = lo + (n - 1) * step + 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// CTA (blockIdx.x, blockIdx.y): a.tok tokens from a.tok * blockIdx.x on, 256
// threads of VEC channels of [x | B | C] each, the last blockIdx.y the dt
// heads. A thread walks its channels' tokens with the three inputs before the
// token in registers. The conv state of a request is read and written by one
// CTA alone, the one that holds the request's first token: it also runs the
// request's second and third token, which read the old state too, when they
// lie past its own tokens (the next CTA leaves them out), and it writes the
// state's new rows, the request's last three inputs, from the projection's
// rows. Each input row is read once plus three rows of a CTA's tokens before
// (from L2), each output written once. Four channels per thread come through
// shared memory, 8 bytes of each row by the thread that works on them, a group
// of four rows at work and two on their way; three CTAs of 80 registers per SM
// (four of 64 spill: 0.660 ms for the case below, but 42 us for 16 prompts of 1
// to 1501 tokens, where three take 38 us). B200, 256 prompts of 512 tokens,
// 6144 channels (3.29 GB): 0.657 ms in bursts, 0.76 of the copy rate (0.69 to
// 0.73 ms back to back); 0.71 ms with the next rows in registers, 0.77 ms with
// eight channels. No pipe is full (issue, 18 instructions per element, is 61 %
// busy): what is left is the dependences of the 24 warps that an SM holds. One
// channel per thread (counts that are no multiples of 4): 64 prompts of 512
// tokens, 63 heads, 0.76 ms, 0.17 of the copy rate.
// ---------------------------------------------------------------------------
// What a thread of k_conv_prompt has of its channels: VEC as one load brings
// them, as floats, and the products.
template <int VEC> struct Chans;
template <> struct Chans<4> {
    using Raw = uint2;
    float2 f[2];
    __device__ __forceinline__ void set(const Raw& u) {
        f[0] = make_float2(bf_lo(u.x), bf_hi(u.x));
        f[1] = make_float2(bf_lo(u.y), bf_hi(u.y));
    }
};
template <> struct Chans<1> {
    using Raw = uint16_t;
    float2 f[1];
    __device__ __forceinline__ void set(const Raw& u) { f[0] = make_float2(bf_lo(u), 0.f); }
};

template <int VEC>
__global__ void __launch_bounds__(kConvThreads, 3) k_conv_prompt(const ConvPromptArgs a) {
    using Raw = typename Chans<VEC>::Raw;
    constexpr int kPairs = (VEC + 1) / 2;
    constexpr int kAhead = 4;  // rows fetched together
    constexpr int kRing = 3;   // such groups, one at work
    const int chans = a.din + 2 * a.gn;
    const size_t Dp = static_cast<size_t>(a.din) + chans + a.H;
    const int t0 = blockIdx.x * a.tok, t1 = min(a.total - t0, a.tok) + t0;
    if (blockIdx.x == 0 && blockIdx.y == 0)  // every range, those without a token here too
        for (int r = threadIdx.x; r < a.batch; r += kConvThreads)
            if (a.cu[r] < 0 || a.cu[r + 1] < a.cu[r] || a.cu[r + 1] > a.total) set_error(a.err, RSSM_DEVERR_SEQ_RANGE);
    const int request0 = first_request(a.cu, a.batch, t0);
    if (blockIdx.y == gridDim.y - 1) {  // dt
        for (int r = request0; r < a.batch; ++r) {
            const int s = a.cu[r], e = a.cu[r + 1];
            if (s >= t1) break;
            if (s < 0 || e < s || e > a.total) continue;
            const int from = max(s, t0), to = min(e, t1);
            // (256 tokens of 2^23 heads are 2^31 values)
            const unsigned n = to > from ? static_cast<unsigned>(to - from) * a.H : 0u;
            for (unsigned i = threadIdx.x; i < n; i += kConvThreads) {
                const size_t t = from + i / static_cast<unsigned>(a.H);
                const unsigned h = i % static_cast<unsigned>(a.H);
                const float v = bf(a.zx[t * Dp + a.din + chans + h]) + a.dt_bias[h];
                a.dt[t * a.H + h] = v > 20.0f ? v : log1pf(expf(v));
            }
        }
        return;
    }
    const int c = VEC * (blockIdx.y * kConvThreads + threadIdx.x);
    if (c >= chans) return;
    float2 w[kTaps][kPairs], bias[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int c1 = c + 2 * i + (VEC > 1);  // (VEC 1: the pair's second half is not used)
        const float4 v0 = reinterpret_cast<const float4*>(a.w)[c + 2 * i], v1 = reinterpret_cast<const float4*>(a.w)[c1];
        w[0][i] = make_float2(v0.x, v1.x);
        w[1][i] = make_float2(v0.y, v1.y);
        w[2][i] = make_float2(v0.z, v1.z);
        w[3][i] = make_float2(v0.w, v1.w);
        bias[i] = make_float2(a.bias[c + 2 * i], a.bias[c1]);
    }
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
    __shared__ Raw ring[VEC == 4 ? kRing * kAhead * kConvThreads : 1];
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring + threadIdx.x));
    auto row = [&](int t) { return *reinterpret_cast<const Raw*>(in + static_cast<size_t>(t) * Dp); };
    for (int r = request0; r < a.batch; ++r) {
        const int s = a.cu[r], e = a.cu[r + 1];
        if (s >= t1) break;
        if (s < 0 || e <= s || e > a.total) continue;
        const bool first = s >= t0;
        const int from = first ? s : max(t0, s + kTaps - 1);
        const int to = first ? max(min(e, t1), min(e, s + kTaps - 1)) : min(e, t1);
        Chans<VEC> r0, r1, r2;  // the three inputs before the token
        if (first) {
            __nv_bfloat16* st = a.state + static_cast<size_t>(r) * (kTaps - 1) * chans + c;
            Raw* s0 = reinterpret_cast<Raw*>(st);
            Raw* s1 = reinterpret_cast<Raw*>(st + chans);
            Raw* s2 = reinterpret_cast<Raw*>(st + 2 * static_cast<size_t>(chans));
            const Raw o0 = *s0, o1 = *s1, o2 = *s2;
            r0.set(o0);
            r1.set(o1);
            r2.set(o2);
            // the last three inputs of the request, or of the old state
            const int n = e - s;
            *s0 = n >= 3 ? row(e - 3) : n == 2 ? o2 : o1;
            *s1 = n >= 2 ? row(e - 2) : o2;
            *s2 = row(e - 1);
        } else if (from < to) {
            r0.set(row(from - 3));
            r1.set(row(from - 2));
            r2.set(row(from - 1));
        }
        const __nv_bfloat16* from_x = in + static_cast<size_t>(from) * Dp;   // the next row to fetch
        __nv_bfloat16* to_y = dst + static_cast<size_t>(from) * width;      // the next token's results
        auto token = [&](const Raw& raw) {
            Chans<VEC> cur;
            cur.set(raw);
            uint32_t y[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                float2 o = fma2(w[0][i], r0.f[i], bias[i]);
                o = fma2(w[1][i], r1.f[i], o);
                o = fma2(w[2][i], r2.f[i], o);
                o = fma2(w[3][i], cur.f[i], o);
                y[i] = silu2(o);
            }
            if constexpr (VEC == 4)
                *reinterpret_cast<uint2*>(to_y) = make_uint2(y[0], y[1]);
            else
                *reinterpret_cast<uint16_t*>(to_y) = static_cast<uint16_t>(y[0]);
            to_y += width;
            r0 = r1;
            r1 = r2;
            r2 = cur;
        };
        if constexpr (VEC == 4) {
            const int n = to - from;
            int got = 0;  // rows fetched, or asked for past the last
            auto fetch = [&](int buf) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (got + k < n)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                                         mine + (buf * kAhead + k) * 8 * kConvThreads),
                                     "l"(from_x)
                                     : "memory");
                    from_x += Dp;
                }
                got += kAhead;
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
#pragma unroll
            for (int i = 0; i < kRing - 1; ++i) fetch(i);
            int buf = 0;
#pragma unroll 1
            for (int i = 0; i < n; i += kAhead) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
                Raw raw[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) raw[k] = ring[(buf * kAhead + k) * kConvThreads + threadIdx.x];
                fetch(buf == 0 ? kRing - 1 : buf - 1);
                buf = buf + 1 == kRing ? 0 : buf + 1;
                if (i + kAhead <= n) {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) token(raw[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (i + k < n) token(raw[k]);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else {  // 2 bytes of a row: by way of registers
            Raw next[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (from + k < to) {
                    next[k] = *reinterpret_cast<const Raw*>(from_x);
                    from_x += Dp;
                }
            int left = to - from;
#pragma unroll 1
            for (; left >= 2 * kAhead; left -= kAhead)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const Raw raw = next[k];
                    next[k] = *reinterpret_cast<const Raw*>(from_x);
                    from_x += Dp;
                    token(raw);
                }
            left -= kAhead;  // rows not yet fetched
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (k < left + kAhead) token(next[k]);
#pragma unroll 1
            for (; left > 0; --left) {
                const Raw raw = *reinterpret_cast<const Raw*>(from_x);
                from_x += Dp;
                token(raw);
            }
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sum over the `warps` warps that share a row (consecutive warps of the CTA);
// red holds one float per warp of the CTA. Every thread of the CTA calls it
// when warps > 1.
__device__ __forceinline__ float row_sum(float v, int warps, float* red) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = warp & ~(warps - 1);
    __syncthreads();  // an earlier sum's readers are done
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += red[first + i];
    return s;
}

// ---------------------------------------------------------------------------
// Gated norm, rows whose groups split into 16-byte pieces: `warps` warps per
// (row, group), up to 16 elements of it per lane in registers (lane l of the
// part takes elements 8 l .. 8 l + 7 and those 256 x warps on), so y and z are
// read once. A team of warps keeps its group, so its weights stay in
// registers, and takes every (teams / G)-th row. The sigmoid is
// rcp(1 + 2^(-z log2 e)) from the approximate instructions, within 2e-6 of
// itself for |z| < 20, far inside the bf16 rounding of the result.
// B200, 131072 rows of 4096 (8 groups; 4.29 GB): 0.69 ms, 0.96 of the copy
// rate; 2.74 ms with one CTA per row and group that reads y and z twice. 64
// registers: 4 CTAs run per SM.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kNormThreads) k_gate_norm_rows(int rows, int gs, int G, int warps, size_t Dp,
                                                                 const float* __restrict__ y,
                                                                 const __nv_bfloat16* __restrict__ zx,
                                                                 const float* __restrict__ nw, float eps,
                                                                 __nv_bfloat16* __restrict__ out) {
    __shared__ float red[kNormThreads / 32];
    const int per_cta = kNormThreads / 32 / warps;
    const long long team0 = static_cast<long long>(blockIdx.x) * per_cta, team = team0 + (threadIdx.x >> 5) / warps;
    const long long teams = static_cast<long long>(gridDim.x) * per_cta;  // a multiple of G
    const int g = static_cast<int>(team % G);
    const int l = threadIdx.x & (32 * warps - 1);
    const size_t din = static_cast<size_t>(gs) * G, off = static_cast<size_t>(g) * gs;
    int at[2];
    bool in[2];
    float4 w[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        at[k] = 8 * (l + 32 * warps * k);
        in[k] = at[k] < gs;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4* p = reinterpret_cast<const float4*>(nw + off + at[k]);
        w[k][0] = in[k] ? p[0] : zero;
        w[k][1] = in[k] ? p[1] : zero;
    }
    const float inv_n = 1.0f / static_cast<float>(gs);
    const long long step = teams / G;
    for (long long row0 = team0 / G; row0 < rows; row0 += step) {
        // every team of the CTA goes round together (row_sum); the last rows may be missing
        const long long row = row0 + (team / G - team0 / G);
        const bool live = row < rows;
        float v[2][8];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
            uint4 z = make_uint4(0, 0, 0, 0);
            if (live && in[k]) {
                const float4* py = reinterpret_cast<const float4*>(y + row * din + off + at[k]);
                a0 = py[0];
                a1 = py[1];
                z = *reinterpret_cast<const uint4*>(zx + row * Dp + off + at[k]);
            }
            const float ya[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float zf = i & 1 ? bf_hi(zw[i / 2]) : bf_lo(zw[i / 2]);
                v[k][i] = ya[i] * (zf * rcp_approx(1.0f + ex2_approx(zf * -1.4426950408889634f)));
                ss = fmaf(v[k][i], v[k][i], ss);
            }
        }
        const float inv = rsqrtf(row_sum(ss, warps, red) * inv_n + eps);
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!in[k]) continue;
            const float ww[8] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w, w[k][1].x, w[k][1].y, w[k][1].z, w[k][1].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = pack_bf16(v[k][2 * i] * inv * ww[2 * i], v[k][2 * i + 1] * inv * ww[2 * i + 1]);
            *reinterpret_cast<uint4*>(out + row * din + off + at[k]) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Any other group size or row stride: one CTA per (row, group), element by
// element, y and z read twice. B200: 65536 rows of 8192 in one group 1.58 ms,
// 0.41 of the copy rate; 133152 rows of 4032 (9 groups, rows that start on 2
// bytes) 2.69 ms, 0.24.
__global__ void __launch_bounds__(kNormThreads) k_gate_norm_any(int gs, int G, size_t Dp, const float* __restrict__ y,
                                                                const __nv_bfloat16* __restrict__ zx,
                                                                const float* __restrict__ nw, float eps,
                                                                __nv_bfloat16* __restrict__ out) {
    __shared__ float red[kNormThreads / 32];
    const size_t row = blockIdx.x, din = static_cast<size_t>(gs) * G;
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
    const float inv = rsqrtf(row_sum(ss, kNormThreads / 32, red) / static_cast<float>(gs) + eps);
    for (int i = threadIdx.x; i < gs; i += kNormThreads)
        out[row * din + off + i] = __float2bfloat16_rn(gated(i) * inv * nw[off + i]);
}

struct AddNormArgs {
    int rows, dim;
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

// Eight consecutive values as they are kept in memory.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load(const uint4* p, int) { u = *p; }  // 16-byte parts so far apart
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
    // elements lo .. hi - 1, where lo is 0 or hi is 8
    __device__ __forceinline__ void store_part(__nv_bfloat16* p, int lo, int hi) const {
        const int n = hi - lo;
        if (n & 4) *reinterpret_cast<uint2*>(p + (lo ? 4 : 0)) = lo ? make_uint2(u.z, u.w) : make_uint2(u.x, u.y);
        const bool far = lo ? !(n & 4) : n & 4;  // what is left lies in the second half
        if (n & 2) {
            const int i = lo ? (n & 4 ? 2 : 6) : n & 4;
            *reinterpret_cast<uint32_t*>(p + i) = lo ? (far ? u.w : u.y) : (far ? u.z : u.x);
        }
        if (n & 1) {
            const int i = lo ? lo : hi - 1;
            const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
            p[i] = __ushort_as_bfloat16(static_cast<uint16_t>(i & 1 ? w >> 16 : w));
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf_lo(w[i]), f[2 * i + 1] = bf_hi(w[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        u = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void load(const uint4* p, int step) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + step);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void store_part(float* p, int lo, int hi) const {  // where lo is 0 or hi is 8
        const int n = hi - lo;
        if (n & 4) *reinterpret_cast<float4*>(p + (lo ? 4 : 0)) = lo ? b : a;
        const bool far = lo ? !(n & 4) : n & 4;  // what is left lies in the second half
        const float4 q = far ? b : a;
        const int base = far ? 4 : 0;
        if (n & 2) *reinterpret_cast<float2*>(p + base + (lo ? 2 : 0)) = lo ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
        if (n & 1) {
            const int i = (lo ? lo : hi - 1) & 3;
            p[base + i] = i < 2 ? (i ? q.y : q.x) : (i > 2 ? q.w : q.z);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return bf(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ---------------------------------------------------------------------------
// Add and norms, dim a multiple of 8: `warps` warps per row, up to 32 elements
// of it per lane in registers (four pieces of 8, 256 x warps apart), so u and
// v are read once and both sums of squares are taken from registers.
// B200, 131072 rows of 2048, bf16 stream, every option (2.15 GB): 0.385 ms,
// 0.85 of the copy rate (0.69 ms with the rows as floats in registers: half
// the warps); fp32 stream (3.22 GB) 0.66 ms, 0.75. Bound by L1 as much as by
// HBM: the weights, 12 bytes an element, come from it for every row (its data
// pipe 78 % busy, DRAM 70 %).
// ---------------------------------------------------------------------------
template <typename TU>
__global__ void __launch_bounds__(512) k_add_norm_rows(const AddNormArgs a, const int warps) {
    __shared__ float red[16];
    const int l = threadIdx.x & (32 * warps - 1);
    const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / 32 / warps) + (threadIdx.x >> 5) / warps;
    const bool live = row < a.rows;
    const float inv_n = 1.0f / static_cast<float>(a.dim);
    const size_t r0 = static_cast<size_t>(live ? row : 0) * a.dim;
    auto at = [&](int k) { return 8 * (l + 32 * warps * k); };
    Eight<TU> u[4];
    Eight<__nv_bfloat16> v[4];
    float f[8], g[8], ss = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        u[k].zero();
        v[k].zero();
        if (live && at(k) < a.dim) {
            u[k].load(static_cast<const TU*>(a.u) + r0 + at(k));
            if (a.v) v[k].load(a.v + r0 + at(k));
        }
    }
    if (a.v) {
        float inv = 1.0f;
        if (a.post_w) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
            }
            inv = rsqrtf(row_sum(ss, warps, red) * inv_n + a.eps);
            ss = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (at(k) >= a.dim) continue;
            Eight<float> c;
            v[k].get(f);
            if (a.post_w) {
                c.load(a.post_w + at(k));
                c.get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * g[i];
            }
            if (a.gate) {
                c.load(a.gate + at(k));
                c.get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= g[i];
            }
            u[k].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmaf(a.scale, f[i], g[i]);
            u[k].set(g);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (a.u_out && live && at(k) < a.dim) u[k].store(static_cast<TU*>(a.u_out) + r0 + at(k));
        u[k].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
    }
    if (!a.out) return;
    const float pre = rsqrtf(row_sum(ss, warps, red) * inv_n + a.eps);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!live || at(k) >= a.dim) continue;
        Eight<float> c;
        c.load(a.pre_w + at(k));
        c.get(g);
        u[k].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * pre * g[i];
        Eight<__nv_bfloat16> o;
        o.set(f);
        o.store(a.out + r0 + at(k));
    }
}

// ---------------------------------------------------------------------------
// Any other width from 9 to kShiftDim: a row starts at any of 8 places in a
// piece of 8 elements (the same one in u, v, u_out and out, which all start on
// 16 bytes), so a team of warps takes rows that many teams apart, a multiple
// of 8: its rows all start at the same place. A lane has one piece of a row (K =
// 2 above 4089 elements: two) with its weights in registers for every row. The
// next two rows are on their way to shared memory, 16 bytes at a time; the
// pieces at a row's ends are stored in parts. No pipe is full (issue was 63 %
// busy before pairs of fp32 went through one instruction): each row waits for
// its two sums.
// B200: 5003 rows of 2561, fp32 stream (154 MB), 41 us, 0.57 of the copy rate;
// 20000 of 2561, bf16, 111 us (0.57); 200000 of 1001, fp32, 0.54 ms (0.69);
// 700000 of 257, bf16, 0.67 ms (0.33); 24000 of 8185, fp32, 0.55 ms (0.66).
// Element by element these took 55, 247, 686, 785 and 1120 us. The next row's
// pieces in registers instead: 57 and 138 us for the first two.
// ---------------------------------------------------------------------------
constexpr int kShiftRows = 3;                      // rows of a team on their way or at work
// Threads per SM in a grid. K = 1 (64 registers) runs them all at once. K = 2
// (128 registers) runs one CTA per SM, and the grid is two or three rounds of
// them: 1 to 5 % faster than one round of many rows, since a CTA's start meets
// another's end (24000 rows of 8185, fp32: 0.565 and 0.585 ms), slower for few
// (300 rows: 23 and 19 us).
constexpr int kShiftHold = 1024;
constexpr int kShiftThreads = 512;
constexpr int kShiftDim = 16 * kShiftThreads - 7;  // two pieces per thread wherever the row starts

// 16 bytes into shared memory, `n` of them read and the rest zeros.
__device__ __forceinline__ void copy16(uint4* dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(n)
                 : "memory");
}

template <typename TU, int K>
__global__ void __launch_bounds__(kShiftThreads) k_add_norm_shifted(const AddNormArgs a, const int warps) {
    // partial sums of the teams' warps, two sets in turn (one barrier per sum)
    __shared__ float4 red[2][8][kShiftThreads / 128];
    extern __shared__ __align__(16) uint4 sm[];  // [kShiftRows][K][u's 16-byte parts, v][threads]
    constexpr int kParts = sizeof(TU) / 2, kPer = 16 / sizeof(TU);  // 16-byte parts of u, elements of one
    const int warp = threadIdx.x >> 5, in_cta = warp / warps, per_cta = blockDim.x / 32 / warps;
    if (threadIdx.x < sizeof(red) / 16) (&red[0][0][0])[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int team = blockIdx.x * per_cta + in_cta, teams = gridDim.x * per_cta;  // a multiple of 8
    const int off = static_cast<int>(static_cast<long long>(team) * a.dim & 7);
    // the pieces' first elements of the row and the parts of them that are the row's
    const int e0 = 8 * (static_cast<int>(threadIdx.x) - 32 * warps * in_cta) - off, apart = 256 * warps;
    int lo[K], hi[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        lo[k] = max(0, -(e0 + k * apart));
        hi[k] = min(8, a.dim - (e0 + k * apart));
    }
    auto inside = [&](int k, int i) { return i >= lo[k] && i < hi[k]; };
    auto whole = [&](int k) { return lo[k] == 0 && hi[k] == 8; };
    const long long step = static_cast<long long>(teams) * a.dim;
    // the pieces of the next row on their way to this thread's places in a
    // buffer, its neighbours' elements too (whatever they are at the time), but
    // nothing past the last row; zeros where there is no row or no piece
    long long next = team, at = static_cast<long long>(team) * a.dim + e0, from = at;
    uint4* const mine = sm + threadIdx.x;
    const int part = blockDim.x, set = (kParts + 1) * part;
    auto fetch = [&](int buf) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int n = 8;  // elements
            if (next + 1 >= a.rows) n = next < a.rows ? hi[k] : 0;
            if (lo[k] >= hi[k]) n = 0;
            const long long i = n ? from + k * apart : 0;
            uint4* to = mine + (buf * K + k) * set;
            copy16(to, static_cast<const TU*>(a.u) + i, min(kPer, n) * static_cast<int>(sizeof(TU)));
            if constexpr (kParts == 2)
                copy16(to + part, static_cast<const TU*>(a.u) + i + (n > kPer ? kPer : 0),
                       max(0, n - kPer) * static_cast<int>(sizeof(TU)));
            if (a.v) copy16(to + kParts * part, a.v + i, 2 * n);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next += teams;
        from += step;
    };
#pragma unroll
    for (int i = 0; i < kShiftRows - 1; ++i) fetch(i);
    float2 post[K][4], pre[K][4];  // post_w times gate; pre_w
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float p[8], q[8];
        const int e = e0 + k * apart;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = a.v && a.post_w && inside(k, i) ? a.post_w[e + i] : 1.f;
            if (a.v && a.gate && inside(k, i)) p[i] *= a.gate[e + i];
            q[i] = a.out && inside(k, i) ? a.pre_w[e + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            post[k][i] = make_float2(p[2 * i], p[2 * i + 1]);
            pre[k][i] = make_float2(q[2 * i], q[2 * i + 1]);
        }
    }
    const float inv_n = 1.0f / static_cast<float>(a.dim);
    const float2 scale = make_float2(a.scale, a.scale);
    const float* sums = reinterpret_cast<const float*>(red[0][in_cta]);
    int turn = 0;
    auto norm = [&](const float2(&f)[K][4]) {  // 1 / sqrt(mean of the row's squares + eps)
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = fma2(f[k][i], f[k][i], s2);
        float v = warp_sum(s2.x + s2.y);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) const_cast<float*>(sums)[turn + warp - in_cta * warps] = v;
            __syncthreads();
            const float4* r = reinterpret_cast<const float4*>(sums + turn);
            v = 0.f;
            for (int i = 0; i < (warps + 3) / 4; ++i) v += (r[i].x + r[i].y) + (r[i].z + r[i].w);
            turn ^= 8 * kShiftThreads / 32;
        }
        return rsqrtf(v * inv_n + a.eps);
    };
    auto pairs = [&](const auto& r, float2(&f)[4]) {
        float g[8];
        r.get(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(g[2 * i], g[2 * i + 1]);
    };
    auto get = [&](const auto& r, int k, float2(&f)[4]) {  // zeros outside the row
        pairs(r, f);
        if (!whole(k))
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = make_float2(inside(k, 2 * i) ? f[i].x : 0.f, inside(k, 2 * i + 1) ? f[i].y : 0.f);
    };
    auto set8 = [&](auto& r, const float2(&f)[4]) {
        const float g[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
        r.set(g);
    };
    auto store = [&](const auto& r, int k, auto* p) {
        if (whole(k))
            r.store(p + at + k * apart);
        else if (lo[k] < hi[k])
            r.store_part(p + at + k * apart, lo[k], hi[k]);
    };
    int buf = 0;
    __syncthreads();  // red is zeros
    for (long long row = team, first = static_cast<long long>(blockIdx.x) * per_cta; first < a.rows;
         first += teams, row += teams, at += step) {  // every team of the CTA goes round together
        asm volatile("cp.async.wait_group %0;" ::"n"(kShiftRows - 2) : "memory");
        Eight<TU> u[K];
        Eight<__nv_bfloat16> v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint4* here = mine + (buf * K + k) * set;
            u[k].load(here, part);
            if (a.v) v[k].load(here + kParts * part, part);
        }
        buf = buf == 0 ? kShiftRows - 1 : buf - 1;  // where the row before was
        fetch(buf);
        buf = buf + 2 >= kShiftRows ? buf + 2 - kShiftRows : buf + 2;
        float2 f[K][4], g[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) get(u[k], k, g[k]);
        if (a.v) {
#pragma unroll
            for (int k = 0; k < K; ++k) get(v[k], k, f[k]);
            const float inv = a.post_w ? norm(f) : 1.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    g[k][i] = fma2(scale, mul2(mul2(f[k][i], make_float2(inv, inv)), post[k][i]), g[k][i]);
                set8(u[k], g[k]);
                if constexpr (kParts == 1) pairs(u[k], g[k]);  // as it is kept
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (a.u_out && row < a.rows) store(u[k], k, static_cast<TU*>(a.u_out));
        if (!a.out) continue;
        const float inv = norm(g);
        if (row >= a.rows) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Eight<__nv_bfloat16> o;
#pragma unroll
            for (int i = 0; i < 4; ++i) g[k][i] = mul2(mul2(g[k][i], make_float2(inv, inv)), pre[k][i]);
            set8(o, g[k]);
            store(o, k, a.out);
        }
    }
}

// The widest and the narrowest rows of other widths: `warps` warps per row,
// element by element, kAddKeep elements per lane in registers and the rest of
// a wide row read again. B200, 3000 rows of 12001, fp32 stream (432 MB): 0.29
// ms, 0.23 of the copy rate.
constexpr int kAddKeep = 12;
template <typename TU>
__global__ void __launch_bounds__(kNormThreads) k_add_norm_any(const AddNormArgs a, const int warps) {
    __shared__ float red[kNormThreads / 32];
    const int l = threadIdx.x & (32 * warps - 1), step = 32 * warps;
    const long long row = static_cast<long long>(blockIdx.x) * (kNormThreads / 32 / warps) + (threadIdx.x >> 5) / warps;
    const int dim = row < a.rows ? a.dim : 0;  // (a team without a row takes part in the sums)
    const size_t r0 = dim ? static_cast<size_t>(row) * a.dim : 0;
    const float inv_n = 1.0f / static_cast<float>(a.dim);
    const TU* u = static_cast<const TU*>(a.u) + r0;
    TU* uo = a.u_out ? static_cast<TU*>(a.u_out) + r0 : nullptr;
    const __nv_bfloat16* v = a.v ? a.v + r0 : nullptr;
    float ku[kAddKeep], kv[kAddKeep];
#pragma unroll
    for (int k = 0; k < kAddKeep; ++k) {
        const int i = l + k * step;
        ku[k] = i < dim ? to_f(u[i]) : 0.f;
        kv[k] = v && i < dim ? bf(v[i]) : 0.f;
    }
    float inv = 1.f;
    if (v && a.post_w) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < kAddKeep; ++k) ss = fmaf(kv[k], kv[k], ss);
        for (int i = l + kAddKeep * step; i < dim; i += step) ss = fmaf(bf(v[i]), bf(v[i]), ss);
        inv = rsqrtf(row_sum(ss, warps, red) * inv_n + a.eps);
    }
    auto stream = [&](int i, float t, float f) {  // u' as it is kept
        if (v) {
            if (a.post_w) f = f * inv * a.post_w[i];
            if (a.gate) f *= a.gate[i];
            t = fmaf(a.scale, f, t);
        }
        TU k;
        put(&k, t);
        return k;
    };
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < kAddKeep; ++k) {
        const int i = l + k * step;
        if (i < dim) {
            const TU t = stream(i, ku[k], kv[k]);
            if (uo) uo[i] = t;
            ku[k] = to_f(t);
        }
        ss = fmaf(ku[k], ku[k], ss);
    }
    for (int i = l + kAddKeep * step; i < dim; i += step) {
        const TU t = stream(i, to_f(u[i]), v ? bf(v[i]) : 0.f);
        if (a.out) ss = fmaf(to_f(t), to_f(t), ss);
        if (uo && !a.out) uo[i] = t;
    }
    if (!a.out) return;
    const float pre = rsqrtf(row_sum(ss, warps, red) * inv_n + a.eps);
#pragma unroll
    for (int k = 0; k < kAddKeep; ++k) {
        const int i = l + k * step;
        if (i < dim) a.out[r0 + i] = __float2bfloat16_rn(ku[k] * pre * a.pre_w[i]);
    }
    for (int i = l + kAddKeep * step; i < dim; i += step) {
        const TU t = stream(i, to_f(u[i]), v ? bf(v[i]) : 0.f);
        if (uo) uo[i] = t;
        a.out[r0 + i] = __float2bfloat16_rn(to_f(t) * pre * a.pre_w[i]);
    }
}

// Streaming multiprocessors of the current device.
int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
    if (dev < 64 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
    if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
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
    if (total < 0 || total > RSSM_PROMPT_TOKENS_MAX || !cu_seqlens || !conv_state || !conv_w || !conv_b || !dt_bias)
        return RSSM_ERR_INVALID_ARG;
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
    // four channels at a time when every row and each of x, B, C starts on 8 bytes
    const int chans = a.din + 2 * a.gn;
    const bool vec = a.din % 4 == 0 && a.gn % 4 == 0 && a.H % 4 == 0;
    const int per_cta = (vec ? 4 : 1) * kConvThreads;
    const int ny = (chans + per_cta - 1) / per_cta + 1;  // and the dt heads
    if (ny > 65535 || a.H > 1 << 23) return RSSM_ERR_SHAPE;  // (a CTA counts its dt values in 32 bits)
    // Tokens per CTA: 256 (three rows before them are read again, and the
    // weights once per CTA; 697 us at 64, 665 us at 128, 657 us at 256 for
    // 256 x 512 tokens), fewer while that leaves SMs without work
    a.tok = 256;
    while (a.tok > 4 && static_cast<long long>((total - 1) / a.tok + 1) * ny < 4ll * sm_count()) a.tok /= 2;
    const dim3 grid(static_cast<unsigned>((total - 1) / a.tok + 1), static_cast<unsigned>(ny));
    if (vec)
        k_conv_prompt<4><<<grid, kConvThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    else
        k_conv_prompt<1><<<grid, kConvThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
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
    const int gs = din / G;
    const __nv_bfloat16* zx = static_cast<const __nv_bfloat16*>(zxbcdt);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // 16-byte pieces, and a group within 16 elements of each thread of a CTA
    if (gs % 8 == 0 && Dp % 8 == 0 && gs <= 16 * kNormThreads) {
        int warps = 1;
        while (512 * warps < gs) warps *= 2;
        const int per_cta = kNormThreads / 32 / warps;  // teams
        // teams a multiple of G (a team keeps its group): whole rounds of G CTAs
        // or, when a CTA has a multiple of G teams, any number of CTAs; no more
        // than there are rows or 8 per SM, twice what runs at once (with 4 per
        // SM: 0.663 ms for 131072 rows of 4096 in bursts either way, 17.4 us
        // instead of 19.0 for 3000)
        const long long unit = per_cta % G == 0 ? 1 : G, rows_per_unit = unit * per_cta / G;
        const long long want = (rows + rows_per_unit - 1) / rows_per_unit;
        const long long hold = 8ll * sm_count() / unit;
        const long long units = want < hold ? want : hold > 0 ? hold : 1;
        k_gate_norm_rows<<<static_cast<unsigned>(units * unit), kNormThreads, 0, st>>>(rows, gs, G, warps, Dp, y, zx,
                                                                                       norm_w, eps, o);
        return launched();
    }
    if (G > 65535) return RSSM_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(G));
    k_gate_norm_any<<<grid, kNormThreads, 0, st>>>(gs, G, Dp, y, zx, norm_w, eps, o);
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
    a.rows = rows;
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dim % 8 == 0) {
        int warps = 1;  // per row, 1024 elements each
        while (1024 * warps < dim) warps *= 2;
        const int threads = warps > 8 ? 32 * warps : 256, per_cta = threads / 32 / warps;
        const unsigned grid = static_cast<unsigned>((rows - 1) / per_cta + 1);
        if (u_dtype == RSSM_F32)
            k_add_norm_rows<float><<<grid, threads, 0, st>>>(a, warps);
        else
            k_add_norm_rows<__nv_bfloat16><<<grid, threads, 0, st>>>(a, warps);
    } else if (dim > 8 && dim <= kShiftDim) {
        const bool two = dim > 8 * kShiftThreads - 7;
        const int warps = (dim + 7 + (two ? 511 : 255)) / (two ? 512 : 256), per_cta = warps < 8 ? 8 / warps : 1;
        const int threads = 32 * warps * per_cta;
        // teams a multiple of 8, no more than kShiftHold threads per SM or there are rows
        const long long unit = per_cta % 8 == 0 ? 1 : per_cta % 4 == 0 ? 2 : per_cta % 2 == 0 ? 4 : 8;
        const long long want = (rows - 1ll + unit * per_cta) / (unit * per_cta);
        const long long hold = static_cast<long long>(sm_count()) * (kShiftHold / threads) / unit;
        const unsigned grid = static_cast<unsigned>(unit * (want < hold ? want : hold > 0 ? hold : 1));
        const size_t piece = u_dtype == RSSM_F32 ? 48 : 32;
        auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
            if (rssm::allow_smem(kernel, kShiftRows * kShiftThreads * 2 * 48, done) != cudaSuccess) return RSSM_ERR_CUDA;
            kernel<<<grid, threads, kShiftRows * threads * piece * (two ? 2 : 1), st>>>(a, warps);
            return launched();
        };
        static std::atomic<uint64_t> done[4];
        if (u_dtype == RSSM_F32)
            return two ? go(k_add_norm_shifted<float, 2>, done[0]) : go(k_add_norm_shifted<float, 1>, done[1]);
        return two ? go(k_add_norm_shifted<__nv_bfloat16, 2>, done[2]) : go(k_add_norm_shifted<__nv_bfloat16, 1>, done[3]);
    } else {
        int warps = 1;  // per row, the elements that lanes keep
        while (warps < kNormThreads / 32 && 32 * kAddKeep * warps < dim) warps *= 2;
        const unsigned grid = static_cast<unsigned>((rows - 1) / (kNormThreads / 32 / warps) + 1);
        if (u_dtype == RSSM_F32)
            k_add_norm_any<float><<<grid, kNormThreads, 0, st>>>(a, warps);
        else
            k_add_norm_any<__nv_bfloat16><<<grid, kNormThreads, 0, st>>>(a, warps);
    }
    return launched();
}

}  // extern "C"
