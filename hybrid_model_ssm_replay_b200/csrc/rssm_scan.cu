// rssm_scan.cu -- the selective scan of packed prompts with its outputs
// (rssm_prefill_scan, include/rssm.h). Per request and head, over the
// request's tokens,
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t,
// from the checkpoint in the head's record and back into it.
//
// Work items. A request runs whole, one CTA per head, when the batch fills
// the GPU. Else its tokens are cut into segments of seg_len tokens: one pass
// forms every segment's state from zero (all but the last segment's), one
// joins them, init_{s+1} = exp(A S_s) init_s + local_s, and one runs every
// segment from its joined state with outputs. Segment s of request b has the
// workspace slot floor(cu[b] / seg_len) + b + s: a request has at most
// floor(cu[b+1] / seg_len) - floor(cu[b] / seg_len) + 1 segments, so slots
// never meet, and there are at most floor(total / seg_len) + batch of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rssm.h"
#include "rssm_device.cuh"
#include "rssm_internal.h"

namespace rssm {

namespace {

// The tokens of request b, [start, end); false (and the error word set) when
// cu_seqlens or the request's position is bad. Every CTA of a request
// answers alike, so a bad request is left untouched as a whole.
__device__ __forceinline__ bool request_range(const ScanArgs& a, int b, int& start, int& end) {
    start = a.cu[b];
    end = a.cu[b + 1];
    if (start < 0 || end < start || end > a.total || end - start > a.max_seqlen) {
        if (threadIdx.x == 0) set_error(a.err, RSSM_DEVERR_SEQ_RANGE);
        return false;
    }
    if (a.pos[b] != 0) {
        if (threadIdx.x == 0) set_error(a.err, RSSM_DEVERR_POS_RANGE);
        return false;
    }
    return true;
}

__device__ __forceinline__ int slot_base(const ScanArgs& a, int b, int start) { return start / a.seg_len + b; }

// The request of a segment slot: the last b whose first slot is <= slot.
__device__ __forceinline__ int slot_request(const ScanArgs& a, int slot) {
    int lo = 0, hi = a.s.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int c = a.cu[mid];
        if (c >= 0 && slot_base(a, mid, c) <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// What one CTA runs: tokens [t0, t1) of request b.
struct Item {
    int b, t0, t1;
    int slot;    // segment slot, -1 when the request runs whole
    bool last;   // its end state is the request's
};

// Item `i` (a request, or a segment slot); false when there is nothing to do.
template <bool OUT>
__device__ __forceinline__ bool find_item(const ScanArgs& a, int i, Item& it) {
    int start, end;
    if (a.seg_len == 0) {
        it.b = i;
        if (!request_range(a, i, start, end) || start == end) return false;
        it.t0 = start;
        it.t1 = end;
        it.slot = -1;
        it.last = true;
        return true;
    }
    it.b = slot_request(a, i);
    if (!request_range(a, it.b, start, end)) return false;
    const int seg = i - slot_base(a, it.b, start);
    const long long t0 = start + static_cast<long long>(seg) * a.seg_len;
    if (seg < 0 || t0 >= end) return false;
    it.t0 = static_cast<int>(t0);
    it.t1 = t0 + a.seg_len < end ? it.t0 + a.seg_len : end;
    it.slot = i;
    it.last = it.t1 == end;
    return OUT || !it.last;
}

__device__ __forceinline__ float* head_state(const ScanArgs& a, int b, int h) {
    return reinterpret_cast<float*>(a.record + (static_cast<size_t>(b) * a.s.H + h) * a.rec.bytes);
}

__device__ __forceinline__ float* slot_state(const ScanArgs& a, int slot, int h) {
    return a.ws + (static_cast<size_t>(slot) * a.s.H + h) * a.s.P * a.s.N;
}

__host__ __device__ __forceinline__ int scan_slots(const ScanArgs& a) { return a.total / a.seg_len + a.s.batch; }

__device__ __forceinline__ float* slot_dtsum(const ScanArgs& a, int slot, int h) {
    return a.ws + static_cast<size_t>(scan_slots(a)) * a.s.H * a.s.P * a.s.N + static_cast<size_t>(slot) * a.s.H + h;
}

// ---------------------------------------------------------------------------
// k_scan: the recurrence token by token, for every shape and both input
// types. One CTA per (item, head); the state stays in registers, lane group
// of N / 4 lanes per state row, 4 columns per lane, PASS rows per thread;
// tokens are staged 16 at a time in shared memory as fp32.
// ---------------------------------------------------------------------------
constexpr int kScanTok = 16;

template <typename TIn, int PASS, bool OUT>
__global__ void __launch_bounds__(kThreads) k_scan(const ScanArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float s_dt[kScanTok];
    const int H = a.s.H, P = a.s.P, N = a.s.N, G = a.s.G, lpr = a.s.lpr;
    const int h = blockIdx.x % H;
    Item it;
    if (!find_item<OUT>(a, blockIdx.x / H, it)) return;
    const int g = h / (H / G), tid = threadIdx.x;
    float* s_x = sm;                          // [kScanTok][P]
    float* s_y = s_x + kScanTok * P;          // [kScanTok][P]
    float* s_B = s_y + kScanTok * P;          // [kScanTok][N]
    float* s_C = s_B + kScanTok * N;          // [kScanTok][N]
    const int col = 4 * (tid & (lpr - 1)), row0 = tid / lpr, step = kThreads / lpr;
    const float* init = it.slot < 0 ? head_state(a, it.b, h) : slot_state(a, it.slot, h);
    float4 st[PASS];
#pragma unroll
    for (int k = 0; k < PASS; ++k) {
        const int p = row0 + k * step;
        st[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (OUT && p < P) st[k] = *reinterpret_cast<const float4*>(init + static_cast<size_t>(p) * N + col);
    }
    const float Ah = a.A[h], Dh = OUT ? a.D[h] : 0.f;
    const TIn* x = static_cast<const TIn*>(a.x);
    const TIn* B = static_cast<const TIn*>(a.B);
    const TIn* C = static_cast<const TIn*>(a.C);
    float dtsum = 0.f;
    for (int t0 = it.t0; t0 < it.t1; t0 += kScanTok) {
        const int T = min(kScanTok, it.t1 - t0);
        __syncthreads();
        for (int i = tid; i < T * P; i += kThreads)
            s_x[i] = to_f32(x[(static_cast<size_t>(t0 + i / P) * H + h) * P + i % P]);
        for (int i = tid; i < T * N; i += kThreads) {
            const size_t at = (static_cast<size_t>(t0 + i / N) * G + g) * N + i % N;
            s_B[i] = to_f32(B[at]);
            if (OUT) s_C[i] = to_f32(C[at]);
        }
        if (tid < T) s_dt[tid] = a.dt[static_cast<size_t>(t0 + tid) * H + h];
        __syncthreads();
        for (int t = 0; t < T; ++t) {
            const float d = s_dt[t], dec = expf(d * Ah);
            dtsum += d;
            const float4 b4 = *reinterpret_cast<const float4*>(s_B + t * N + col);
            float4 c4 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (OUT) c4 = *reinterpret_cast<const float4*>(s_C + t * N + col);
#pragma unroll
            for (int k = 0; k < PASS; ++k) {
                const int p = row0 + k * step;
                const float xp = p < P ? s_x[t * P + p] : 0.f, w = d * xp;
                st[k].x = fmaf(dec, st[k].x, w * b4.x);
                st[k].y = fmaf(dec, st[k].y, w * b4.y);
                st[k].z = fmaf(dec, st[k].z, w * b4.z);
                st[k].w = fmaf(dec, st[k].w, w * b4.w);
                if (OUT) {
                    const float v = group_sum(dot4(st[k], c4), lpr);
                    if (p < P && (tid & (lpr - 1)) == 0) s_y[t * P + p] = fmaf(Dh, xp, v);
                }
            }
        }
        if (OUT) {
            __syncthreads();
            for (int i = tid; i < T * P; i += kThreads)
                a.y[(static_cast<size_t>(t0 + i / P) * H + h) * P + i % P] = s_y[i];
        }
    }
    if (OUT && !it.last) return;
    float* out = OUT ? head_state(a, it.b, h) : slot_state(a, it.slot, h);
#pragma unroll
    for (int k = 0; k < PASS; ++k) {
        const int p = row0 + k * step;
        if (p < P) *reinterpret_cast<float4*>(out + static_cast<size_t>(p) * N + col) = st[k];
    }
    if (!OUT && tid == 0) *slot_dtsum(a, it.slot, h) = dtsum;
}

// ---------------------------------------------------------------------------
// k_scan_join: the segments' start states, in place of their local states.
// One thread per 4 state elements of a (request, head).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) k_scan_join(const ScanArgs a) {
    const int b = blockIdx.x / a.s.H, h = blockIdx.x - b * a.s.H;
    const int i = blockIdx.y * kThreads + threadIdx.x;
    int start, end;
    if (!request_range(a, b, start, end) || start == end) return;
    if (4 * i >= a.s.P * a.s.N) return;
    const int base = slot_base(a, b, start), nseg = (end - start + a.seg_len - 1) / a.seg_len;
    const float Ah = a.A[h];
    float4 carry = reinterpret_cast<const float4*>(head_state(a, b, h))[i];
    for (int s = 0; s < nseg; ++s) {
        float4* p = reinterpret_cast<float4*>(slot_state(a, base + s, h)) + i;
        if (s + 1 == nseg) {
            *p = carry;
            break;
        }
        const float4 add = *p;
        const float dec = expf(Ah * *slot_dtsum(a, base + s, h));
        *p = carry;
        carry = make_float4(fmaf(dec, carry.x, add.x), fmaf(dec, carry.y, add.y), fmaf(dec, carry.z, add.z),
                            fmaf(dec, carry.w, add.w));
    }
}

template <typename TIn, bool OUT>
cudaError_t launch_pass(const ScanArgs& a, int items, cudaStream_t st) {
    const size_t smem = 4u * kScanTok * (2 * static_cast<size_t>(a.s.P) + 2 * static_cast<size_t>(a.s.N));
    const int passes = (a.s.P * a.s.lpr + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(items) * static_cast<unsigned>(a.s.H));
    if (passes <= 1)
        k_scan<TIn, 1, OUT><<<grid, kThreads, smem, st>>>(a);
    else if (passes <= 4)
        k_scan<TIn, 4, OUT><<<grid, kThreads, smem, st>>>(a);
    else if (passes <= 8)
        k_scan<TIn, 8, OUT><<<grid, kThreads, smem, st>>>(a);
    else
        k_scan<TIn, 16, OUT><<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

int scan_segment_len(const Shape& s, int in_bf16, int total, int max_seqlen) {
    (void)in_bf16;
    // CTAs that fill the GPU; whole requests when there are that many, or
    // when the longest is short next to the rest of the work
    const long long fill = 4 * 148;
    const long long share = static_cast<long long>(total) * s.H / fill;  // tokens per CTA, evenly cut
    if (max_seqlen <= 256 || max_seqlen <= 2 * share) return 0;
    const long long len = share < 128 ? 128 : (share + 127) / 128 * 128;
    if ((total / len + s.batch) * s.H > 0x7fffffffLL) return 0;  // one CTA per slot and head
    return static_cast<int>(len);
}

size_t scan_workspace_bytes(const Shape& s, int total, int seg_len) {
    if (seg_len == 0) return 0;
    const size_t slots = static_cast<size_t>(total / seg_len) + s.batch;
    return slots * s.H * (static_cast<size_t>(s.P) * s.N + 1) * sizeof(float);
}

cudaError_t launch_scan(const ScanArgs& a, int in_bf16, cudaStream_t st) {
    if (a.seg_len == 0)
        return in_bf16 ? launch_pass<__nv_bfloat16, true>(a, a.s.batch, st) : launch_pass<float, true>(a, a.s.batch, st);
    const int slots = scan_slots(a);
    cudaError_t e = in_bf16 ? launch_pass<__nv_bfloat16, false>(a, slots, st) : launch_pass<float, false>(a, slots, st);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.s.batch) * static_cast<unsigned>(a.s.H),
                    static_cast<unsigned>((a.s.P * a.s.N / 4 + kThreads - 1) / kThreads));
    k_scan_join<<<grid, kThreads, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return in_bf16 ? launch_pass<__nv_bfloat16, true>(a, slots, st) : launch_pass<float, true>(a, slots, st);
}

}  // namespace rssm
