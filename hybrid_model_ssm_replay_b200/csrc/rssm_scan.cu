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
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

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

// Two fp32 lanes in one instruction.
#define RSSM_F32X2(name, op)                                                       \
    __device__ __forceinline__ float2 name(float2 a, float2 b) {                   \
        float2 d;                                                                  \
        asm("{\n\t.reg .b64 ra, rb, rd;\n\t"                                       \
            "mov.b64 ra, {%2, %3};\n\t"                                            \
            "mov.b64 rb, {%4, %5};\n\t" op                                         \
            " rd, ra, rb;\n\t"                                                     \
            "mov.b64 {%0, %1}, rd;\n\t}"                                           \
            : "=f"(d.x), "=f"(d.y)                                                 \
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                             \
        return d;                                                                  \
    }
RSSM_F32X2(add2, "add.rn.f32x2")
RSSM_F32X2(sub2, "sub.rn.f32x2")
RSSM_F32X2(mul2, "mul.rn.f32x2")
#undef RSSM_F32X2

// ---------------------------------------------------------------------------
// k_scan: the recurrence token by token, for every shape and both input
// types. One CTA per (item, head); the state stays in registers, lane group
// of N / 4 lanes per state row, 4 columns per lane, PASS rows per thread;
// tokens are staged 16 at a time in shared memory as fp32, the next ones
// while these are worked on, and worked on 4 at a time, with the sums of
// their rows shared out over the lanes (31 shuffles for 32 sums). Bound by
// instruction issue. B200, fp32, 32 prompts of 300 tokens, 64 heads of
// 64 x 128: 2.07 ms with a shuffle per row and token and scalar FMAs, 1.22 ms
// as it is.
// ---------------------------------------------------------------------------
constexpr int kScanTok = 16;

// One step of a sum over lanes of several values side by side: lanes `off`
// apart share out the V values, each keeps the sums of half of them (the
// lane with the bit `off` the second half). V = 1: both keep it.
template <int V, int M>
__device__ __forceinline__ void share_sums(float (&v)[M], int off) {
    if constexpr (V == 1) {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    } else {
        const bool up = threadIdx.x & off;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float send = up ? v[i] : v[i + V / 2], keep = up ? v[i + V / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
}

template <typename TIn, int PASS, bool OUT>
__global__ void __launch_bounds__(kThreads) k_scan(const ScanArgs a) {
    extern __shared__ __align__(16) float sm[];
    const int H = a.s.H, P = a.s.P, N = a.s.N, G = a.s.G, lpr = a.s.lpr;
    const int h = blockIdx.x % H;
    Item it;
    if (!find_item<OUT>(a, blockIdx.x / H, it)) return;
    const int g = h / (H / G), tid = threadIdx.x;
    // two buffers of [dt, decay | x | B | C] of kScanTok tokens, and the outputs
    const int xs = (P + 3) & ~3, buf = kScanTok * (2 + xs + 2 * N);
    float* s_y = sm + 2 * buf;  // [kScanTok][P]
    const int col = 4 * (tid & (lpr - 1)), row0 = tid / lpr, step = kThreads / lpr;
    const float* init = it.slot < 0 ? head_state(a, it.b, h) : slot_state(a, it.slot, h);
    float2 st[PASS][2];
#pragma unroll
    for (int k = 0; k < PASS; ++k) {
        const int p = row0 + k * step;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (OUT && p < P) v = *reinterpret_cast<const float4*>(init + static_cast<size_t>(p) * N + col);
        st[k][0] = make_float2(v.x, v.y);
        st[k][1] = make_float2(v.z, v.w);
    }
    const float Ah = a.A[h], Dh = OUT ? a.D[h] : 0.f;
    const TIn* x = static_cast<const TIn*>(a.x);
    const TIn* B = static_cast<const TIn*>(a.B);
    const TIn* C = static_cast<const TIn*>(a.C);
    // tokens t0 .. into buffer `to`, zeros past the item's end (a step of
    // zero keeps the state): one token per 16 threads
    auto stage = [&](int t0, float* to) {
        const int s = tid >> 4, l = tid & 15, t = t0 + s;
        const bool in = t < it.t1;
        if (l == 0) {
            const float d = in ? a.dt[static_cast<size_t>(t) * H + h] : 0.f;
            to[s] = d;
            to[kScanTok + s] = in ? expf(d * Ah) : 1.f;
        }
        float* sx = to + 2 * kScanTok + s * xs;
        float* sB = to + kScanTok * (2 + xs) + s * N;
        float* sC = sB + kScanTok * N;
        const TIn* px = x + (static_cast<size_t>(t) * H + h) * P;
        for (int i = l; i < P; i += 16) sx[i] = in ? to_f32(px[i]) : 0.f;
        const size_t at = (static_cast<size_t>(t) * G + g) * N;
        for (int i = l; i < N; i += 16) {
            sB[i] = in ? to_f32(B[at + i]) : 0.f;
            if (OUT) sC[i] = in ? to_f32(C[at + i]) : 0.f;
        }
    };
    float dtsum = 0.f;
    stage(it.t0, sm);
    int cur = 0;
    for (int t0 = it.t0; t0 < it.t1; t0 += kScanTok, cur ^= 1) {
        const int T = min(kScanTok, it.t1 - t0);
        __syncthreads();  // the tokens are in place; the outputs before have left
        if (t0 + kScanTok < it.t1) stage(t0 + kScanTok, sm + (cur ^ 1) * buf);
        const float* s_d = sm + cur * buf;
        const float* s_x = s_d + 2 * kScanTok;
        const float* s_B = s_d + kScanTok * (2 + xs);
        const float* s_C = s_B + kScanTok * N;
#pragma unroll 1
        for (int t4 = 0; t4 < T; t4 += 4) {
            // four tokens: the state's recurrence, then the sums over its rows side
            // by side (value j PASS + k: token j, row k), shared out over the lanes
            constexpr int V = 4 * PASS;
            float part[V];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t4 + j;
                const float d = s_d[t], dec = s_d[kScanTok + t];
                dtsum += d;
                const float2 dec2 = make_float2(dec, dec);
                const float4 b4 = *reinterpret_cast<const float4*>(s_B + t * N + col);
                const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
                float2 c0, c1;
                if (OUT) {
                    const float4 c4 = *reinterpret_cast<const float4*>(s_C + t * N + col);
                    c0 = make_float2(c4.x, c4.y);
                    c1 = make_float2(c4.z, c4.w);
                }
#pragma unroll
                for (int k = 0; k < PASS; ++k) {
                    const int p = row0 + k * step;
                    const float w = p < P ? d * s_x[t * xs + p] : 0.f;
                    const float2 w2 = make_float2(w, w);
                    st[k][0] = fma2(dec2, st[k][0], mul2(w2, b0));
                    st[k][1] = fma2(dec2, st[k][1], mul2(w2, b1));
                    if (OUT) {
                        const float2 y2 = fma2(st[k][0], c0, mul2(st[k][1], c1));
                        part[j * PASS + k] = y2.x + y2.y;
                    }
                }
            }
            if (OUT) {
                auto put = [&](int n, int steps) {  // the n values of this lane after `steps` steps
                    int first = 0;
                    bool mine = true;
                    for (int i = 0, half = V / 2; i < steps; ++i, half /= 2) {
                        if (half) first += tid & (1 << i) ? half : 0;
                        else if (tid & (1 << i)) mine = false;
                    }
                    if (!mine) return;
#pragma unroll
                    for (int i = 0; i < V / 4; ++i) {
                        const int j = (first + i) / PASS, p = row0 + (first + i) % PASS * step;
                        if (i < n && p < P) s_y[(t4 + j) * P + p] = fmaf(Dh, s_x[(t4 + j) * xs + p], part[i]);
                    }
                };
                share_sums<V>(part, 1);
                share_sums<V / 2>(part, 2);
                if (lpr == 4) {
                    put(V / 4, 2);
                } else {
                    share_sums<V / 4>(part, 4);
                    constexpr int V3 = V / 8 ? V / 8 : 1, V4 = V / 16 ? V / 16 : 1, V5 = V / 32 ? V / 32 : 1;
                    if (lpr == 8) {
                        put(V3, 3);
                    } else {
                        share_sums<V3>(part, 8);
                        if (lpr == 16) {
                            put(V4, 4);
                        } else {
                            share_sums<V4>(part, 16);
                            put(V5, 5);
                        }
                    }
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
        if (p < P)
            *reinterpret_cast<float4*>(out + static_cast<size_t>(p) * N + col) =
                make_float4(st[k][0].x, st[k][0].y, st[k][1].x, st[k][1].y);
    }
    if (!OUT && tid == 0) *slot_dtsum(a, it.slot, h) = dtsum;
}

// ---------------------------------------------------------------------------
// k_scan_umma: the scan in blocks of 128 tokens on the 5th-generation tensor
// cores (bf16 inputs, head_dim a multiple of 8). With c_t the log decay from
// the block's start through token t and h the state before the block,
//     y_t  = exp(c_t) C_t h^T + sum_{s <= t} M_ts x_s + D x_t,
//     M_ts = (C_t . B_s) exp(c_t - c_s) dt_s,
//     h   <- exp(c_127) h + sum_s w_s x_s B_s^T,   w_s = dt_s exp(c_127 - c_s),
// four products with K = 128 or d_state. One CTA of 256 threads per (item,
// head, 64 columns of its head_dim), two CTAs per SM; per block:
//   S = C B^T          [128 t x 128 s], C and B as loaded (exact bf16);
//   O = C h^T          [128 t x 64], the state in three bf16 parts;
//   Y = M x            [128 t x 64], M in three parts, built in tensor memory
//                      over S by the threads that own its rows, x as loaded;
//   U = B^T [w x]      [128 n x 192], w x in three parts.
// Thread (warp w, lane l) owns token and state row 32 (w % 4) + l and half
// the columns (w / 4). The state stays in fp32 registers; O is read and
// scaled, with D x added, before Y takes its place in tensor memory; U takes
// M's. 112 KB of shared memory: C, B, x, and one buffer that holds two parts
// of h and then, with half of C's (read by then), the parts of w x. The third
// part of h lies in x's buffer: its product goes first, and x is fetched when
// it has been read (M is built meanwhile). Each part of the next block is
// fetched (TMA) as soon as its buffer has been read; the outputs leave by way
// of x's buffer and C's first half. Rows past the request's end are zeroed in
// x and B.
//
// Decays. No difference of two sums of dt is formed: between two tokens of
// the same 8 the exponent of M is the running sum of dt from s + 1 to t, and
// else M's factor is (end of s's 8 tokens .. t) x (s + 1 .. end of s's 8
// tokens), each the exponential of a sum of terms of one sign.
//
// Precision: a product of bf16 factors is exact in the fp32 sum, and three
// parts leave 2^-26 of M, w x and the state. O adds its smallest part first,
// so that its large sums take d_state / 16 steps. 2-norm of the outputs'
// errors: 1.8e-7 to 2.3e-7 for prompts of 1 to 256 tokens from states of 0.1
// to 10 (the rms of its elements). With the state in two parts (2^-18) that was
// 3.4e-7 to 2.5e-6, the more the larger the state's share, and the time 3 to 6
// % less; the third part's product takes half of that, the rest is x's later
// fetch and the splitting.
//
// What bounds it. B200, 256 prompts of 512 tokens, 64 heads of 64 x 128
// (4.87 GB, 0.74 ms at the copy rate): 2.0 ms in bursts, 2.2 ms back to back
// under the power cap. No pipe is full (16 prompts of 1024 tokens: the tensor
// pipe 38 % busy, the schedulers 49 %, the shared-memory data pipe 67 %, loads
// and stores half of it, the products' operands the other): each CTA is a
// chain of load, S, M, Y, U and state, and two CTAs (all that tensor memory
// and shared memory hold) overlap no more of it. Steps that paid: TMA for the operands, outputs through shared memory and
// TMA instead of a row per lane (a quarter of the time), M's diagonal blocks
// without branches, code short enough for the instruction cache, even shares
// for the warps. Steps that did not: 512 threads at 64 registers (spills go to
// L2, since shared memory leaves no L1), 512 threads alone on an SM (5 % on
// few long prompts).
//
// x is the one raw operand of Y, so M's zeros (s > t) meet every x of the
// block. In a block with a NaN or infinity in x, Y is formed with zeros in
// their place and they are added for t >= s on the CUDA cores, so that no
// output before them changes.
// ---------------------------------------------------------------------------
constexpr int kSuTok = 128;                    // tokens per block
constexpr int kSuThreads = 256;
constexpr int kSuIssuer = 4;                   // two warps with less of M's lower triangle: of the products
constexpr int kSuStorer = 5;                   // and of the second half of Y and C's first block
constexpr uint32_t kSuBlk = kSuTok * 128u;     // 128 rows of 128 bytes, swizzled: 16 KB
constexpr uint32_t kSuB = 0;                   // B rows, two 64-column blocks
constexpr uint32_t kSuX = 2 * kSuBlk;          // h lo; x rows; outputs
constexpr uint32_t kSuR = 3 * kSuBlk;          // h hi, mid; w x hi, mid
constexpr uint32_t kSuC1 = 5 * kSuBlk;         // C columns 64.. ; later w x lo (right behind hi, mid)
constexpr uint32_t kSuC0 = 6 * kSuBlk;         // C columns 0..63; outputs
constexpr uint32_t kSuCol = 7 * kSuBlk;        // float [128]: dt_s exp(decay from s + 1 to the end of its 8 tokens)
constexpr uint32_t kSuSum = kSuCol + 512;      // float [16]: dt sums of 8 tokens each
constexpr uint32_t kSuBar = kSuSum + 64;       // 8 mbarriers, tensor-memory address
constexpr uint32_t kSuSmem = kSuBar + 80;
constexpr uint32_t kSuCols = 256;              // tensor-memory columns
constexpr uint32_t kTmS = 0, kTmLo = 128, kTmY = 192;  // S, then M hi, mid; M lo; O, then Y (U: 0..191)

// Shared-memory matrix descriptor of a 128-byte-swizzled operand: start
// address, leading and stride byte offsets in 16-byte units, version 1.
__device__ __forceinline__ uint64_t su_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kSuBlk >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, bf16 A and B, M = 128.
__host__ __device__ constexpr uint32_t su_idesc(uint32_t n, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

template <uint32_t IDESC>
__device__ __forceinline__ void su_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(IDESC), "r"(accumulate), "r"(0u)
        : "memory");
}

// The A operand from tensor memory.
template <uint32_t IDESC>
__device__ __forceinline__ void su_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(IDESC), "r"(accumulate), "r"(0u)
        : "memory");
}

__device__ __forceinline__ void su_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void su_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void su_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void su_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void su_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 / 8 consecutive 32-bit columns of this thread's row. The values may be
// used after su_wait_ld only.
__device__ __forceinline__ void su_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void su_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void su_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void su_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void su_ld1(uint32_t taddr, uint32_t& r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

__device__ __forceinline__ float su_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    return d;
}

// A pair of bf16 with zeros in the place of NaN and infinities.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    const uint32_t lo = (w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu;
    return lo | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}

// Two fp32 values as bf16 pairs hi + mid + lo (each the nearest bf16 of what
// the parts before leave; the differences are exact).
__device__ __forceinline__ void split3(float2 v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(v);
    const float2 r = sub2(v, bf2(hi));
    mid = pack_bf16(r);
    lo = pack_bf16(sub2(r, bf2(mid)));
}

// A box of a tensor map (columns from x, token rows from y) into shared memory.
__device__ __forceinline__ void su_tma(uint32_t dst, const CUtensorMap& map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(&map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// One lane of a warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 32 fp32 columns from x of head h, 128 tokens from t, out of shared memory;
// what lies past the tensor is not written.
__device__ __forceinline__ void su_tma_store(const CUtensorMap& map, uint32_t src, int x, int h, int t) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(&map), "r"(src),
                 "r"(x), "r"(h), "r"(t)
                 : "memory");
}

// The same box into L2 only.
__device__ __forceinline__ void su_prefetch(const CUtensorMap& map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(&map), "r"(x), "r"(y) : "memory");
}

// A bounded wait for phase `parity`; the loop of the rare long wait is kept
// out of the kernel's body, which is long enough for the instruction cache.
__device__ __noinline__ bool su_wait_long(uint32_t bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, kWaitNs);
}
__device__ __forceinline__ bool su_wait(uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity, 100000u) || su_wait_long(bar, parity);
}

template <bool OUT>
__global__ void __launch_bounds__(kSuThreads, 2)
    k_scan_umma(const ScanArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my, const int slices) {
    extern __shared__ __align__(1024) unsigned char smem[];  // the swizzled operands lie on 1024-byte boundaries
    const int H = a.s.H, P = a.s.P, N = a.s.N, G = a.s.G;
    const int hs = blockIdx.x % (H * slices), h = hs / slices, p0 = 64 * (hs - h * slices);
    Item it;
    if (!find_item<OUT>(a, blockIdx.x / (H * slices), it)) return;
    const int g = h / (H / G), tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int q = warp & 3, half = warp >> 2;  // rows 32 q .., half the columns
    const int row = 32 * q + lane;          // this thread's token and state row
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_in = sb + kSuBar, bar_s = bar_in + 8, bar_o = bar_in + 16, bar_y = bar_in + 24,
                   bar_u = bar_in + 32, bar_x = bar_in + 40, bar_f = bar_in + 48, bar_l = bar_in + 56;
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(smem + kSuBar + 64);
    const bool wide = N > 64;  // B and C have a second block of 64 columns
    const uint32_t in_bytes = kSuBlk * (wide ? 2u : 1u) * (OUT ? 2u : 1u);  // B and C
    const int xx = h * P + p0, bx = g * N;
    const bool issuer = warp == kSuIssuer;  // its elected lane issues every copy and product
    auto load_c0 = [&](int t) { su_tma(sb + kSuC0, mc, bx, t, bar_in); };
    auto load_x = [&](int t) {
        mbar_expect_tx(bar_x, kSuBlk);
        su_tma(sb + kSuX, mx, xx, t, bar_x);
    };
    auto load_bc = [&](int t) {
        su_tma(sb + kSuB, mb, bx, t, bar_in);
        if (wide) su_tma(sb + kSuB + kSuBlk, mb, bx + 64, t, bar_in);
        if (OUT && wide) su_tma(sb + kSuC1, mc, bx + 64, t, bar_in);
    };
    if (issuer && elect_one()) {
        for (int i = 0; i < 8; ++i) mbar_init(bar_in + 8 * i, 1);
        mbar_expect_tx(bar_in, in_bytes);
        if (OUT) load_c0(it.t0);
        load_bc(it.t0);
        if (OUT)
            su_prefetch(mx, xx, it.t0);
        else
            load_x(it.t0);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + kSuBar + 64),
                     "r"(kSuCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const float* dtg = a.dt + h;
    auto load_dt = [&](int t0) { return t0 + row < it.t1 ? dtg[static_cast<size_t>(t0 + row) * H] : 0.f; };
    float d = load_dt(it.t0);
    // decays as powers of two; finite, so that a step of zero keeps all even then
    const float A2 = a.A[h] * 1.4426950408889634f < -3e38f ? -3e38f : a.A[h] * 1.4426950408889634f;
    const float Dh = OUT ? a.D[h] : 0.f;

    // the state: row `row` (d_state), columns 32 half .. + 31 of the head_dim slice
    float2 hst[16];
    const float* init = it.slot < 0 ? head_state(a, it.b, h) : slot_state(a, it.slot, h);
    const int pb = p0 + 32 * half;  // this thread's first column
    auto init_at = [&](int j) { return OUT && row < N && pb + j < P ? init[static_cast<size_t>(pb + j) * N + row] : 0.f; };
#pragma unroll
    for (int j = 0; j < 16; ++j) hst[j] = make_float2(init_at(2 * j), init_at(2 * j + 1));

    // 16-byte chunk j of this thread's row in a buffer
    auto chunk = [&](uint32_t buf, int j) {
        return reinterpret_cast<uint4*>(smem + buf + row * 128 + 16 * (j ^ (row & 7)));
    };
    auto put_state = [&]() {  // hi, mid and lo parts of the state, d_state row by row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split3(hst[4 * j + i], hi[i], mid[i], lo[i]);
            *chunk(kSuR, 4 * half + j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *chunk(kSuR + kSuBlk, 4 * half + j) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
            *chunk(kSuX, 4 * half + j) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    };
    // decays of this thread's token within its group of 8, from d
    float* s_col = reinterpret_cast<float*>(smem + kSuCol);
    const int oct = lane >> 3;
    float pre;  // dt sum from the group's start to the token
    auto scan_dt = [&]() {
        float suf = d;  // to the group's end
        pre = d;
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            const float u = __shfl_up_sync(0xffffffffu, pre, off, 8), v = __shfl_down_sync(0xffffffffu, suf, off, 8);
            if ((lane & 7) >= off) pre += u;
            if ((lane & 7) + off < 8) suf += v;
        }
        const float next = __shfl_down_sync(0xffffffffu, suf, 1, 8);
        if (half == 0) {
            s_col[row] = d * su_exp2(A2 * ((lane & 7) == 7 ? 0.f : next));
            if ((lane & 7) == 0) reinterpret_cast<float*>(smem + kSuSum)[4 * q + oct] = suf;
        }
    };
    if (OUT) put_state();
    scan_dt();
    su_fence_before();
    __syncthreads();
    su_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, *s_tmem, 0);
    const uint32_t tml = tm + (static_cast<uint32_t>(32 * q) << 16);  // this warp's lanes
    float dtsum = 0.f;
    bool timed_out = false;

    int par = 0;
    for (int t0 = it.t0; t0 < it.t1; t0 += kSuTok, par ^= 1) {
        const bool more = t0 + kSuTok < it.t1;
        const float dn = more ? load_dt(t0 + kSuTok) : 0.f;
        if (!su_wait(bar_in, par)) timed_out = true;
        if (!more && t0 + row >= it.t1) {  // rows of the next request, or of none
            const uint4 zero = make_uint4(0, 0, 0, 0);
            if (wide || half == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) *chunk(kSuB + half * kSuBlk, j) = zero;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        su_fence_before();
        if (__syncthreads_or(timed_out)) {  // (x, where its copy is under way, lands before the CTA ends)
            if (!OUT) su_wait_long(bar_x, par);
            break;
        }
        // the block, its decays and the state's parts are in place
        su_fence_after();
        if (OUT && issuer) {
            const uint64_t dB = su_desc(sb + kSuB), dR = su_desc(sb + kSuR), dX = su_desc(sb + kSuX);
            const uint64_t dC0 = su_desc(sb + kSuC0), dC1 = su_desc(sb + kSuC1);
            auto state_part = [&](uint64_t part, uint32_t add) {  // O, or more of it
#pragma unroll 1
                for (int ks = 0; ks < N / 16; ++ks)
                    su_mma<su_idesc(64, 0, 1)>(tm + kTmY, (ks < 4 ? dC0 : dC1) + 2 * (ks & 3), part + 128 * ks,
                                               add | (ks > 0));
            };
            if (elect_one()) {
                state_part(dX, 0);  // the smallest part first: the large sums take the fewest steps
                su_commit(bar_l);
#pragma unroll 1
                for (int ks = 0; ks < N / 16; ++ks)
                    su_mma<su_idesc(128, 0, 0)>(tm + kTmS, (ks < 4 ? dC0 : dC1) + 2 * (ks & 3),
                                                dB + (ks >> 2) * (kSuBlk / 16) + 2 * (ks & 3), ks > 0);
                su_commit(bar_s);
                state_part(dR + kSuBlk / 16, 1);
                state_part(dR, 1);
                su_commit(bar_o);
                if (more) {  // the next block on its way to L2
                    su_prefetch(mx, xx, t0 + kSuTok);
                    su_prefetch(mb, bx, t0 + kSuTok);
                    su_prefetch(mc, bx, t0 + kSuTok);
                    if (wide) su_prefetch(mb, bx + 64, t0 + kSuTok);
                    if (wide) su_prefetch(mc, bx + 64, t0 + kSuTok);
                }
            }
            __syncwarp();
            if (!su_wait(bar_l, par)) timed_out = true;
            if (elect_one()) load_x(t0);  // in the place of the state's lo part
            __syncwarp();
        }
        const float4* s_sum = reinterpret_cast<const float4*>(smem + kSuSum);
        auto sum4 = [&](int i) { return (s_sum[i].x + s_sum[i].y) + (s_sum[i].z + s_sum[i].w); };
        const float4 sums = make_float4(sum4(0), sum4(1), sum4(2), sum4(3));  // of the 32-blocks' dt
        const float total = sums.x + sums.y + sums.z + sums.w;

        // chunk j of x of this block's token s, as given
        auto x_given = [&](int s, int j) {
            if (t0 + s >= it.t1 || p0 + 8 * j >= P) return make_uint4(0, 0, 0, 0);
            return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) +
                                                   (static_cast<size_t>(t0 + s) * H + h) * P + p0 + 8 * j);
        };
        if (OUT) {
            // dt sums from the start of this thread's token's 32-block to the token
            // and of the 32-blocks before
            const float4 mine = s_sum[q];
            const float pre32 = pre + ((oct > 0 ? mine.x : 0.f) + (oct > 1 ? mine.y : 0.f) + (oct > 2 ? mine.z : 0.f));
            const float before = (q > 0 ? sums.x : 0.f) + (q > 1 ? sums.y : 0.f) + (q > 2 ? sums.z : 0.f);
            // M over S, columns 16 half .. + 15 of each of its 32-blocks: hi and mid
            // parts in the columns read, lo in its own
            auto put_m = [&](int J, const float2 (&m)[8]) {
                uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split3(m[i], hi[i], mid[i], lo[i]);
                const uint32_t at = 32 * J + 16 * half;
                su_st8(tml + kTmS + at, hi);
                su_st8(tml + kTmS + at + 8, mid);
                su_st8(tml + kTmLo + at / 2, lo);
            };
            // their column factors in 32-block J; f0, f1: decay from the end of their
            // two groups of 8 to this token
            auto factors = [&](int J, float f0, float f1, float2 (&m)[8]) {
                const float4* c4 = reinterpret_cast<const float4*>(s_col + 32 * J + 16 * half);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 c = c4[i];
                    const float2 f2 = i < 2 ? make_float2(f0, f0) : make_float2(f1, f1);
                    m[2 * i] = mul2(f2, make_float2(c.x, c.y));
                    m[2 * i + 1] = mul2(f2, make_float2(c.z, c.w));
                }
            };
            // the block on the diagonal: factors from the running sum, A2 times the
            // dt sum from s + 1 to t, downwards from the last column; zero for later
            // tokens (whose S may be NaN)
            float f[16];
            {
                float run = half || oct < 2 ? 0.f : A2 * (pre + (oct > 2 ? mine.z : 0.f));
                float dnx = 0.f;
#pragma unroll
                for (int j = 15; j >= 0; --j) {
                    const float ds = __shfl_sync(0xffffffffu, d, 16 * half + j);
                    run = fmaf(A2, lane > 16 * half + j ? dnx : 0.f, run);
                    dnx = ds;
                    f[j] = ds * su_exp2(run);
                }
            }
            if (!su_wait(bar_s, par)) timed_out = true;
            su_fence_after();
            {
                uint32_t v[16];
                su_ld16(tml + kTmS + 32 * q + 16 * half, v);
                su_wait_ld();
                float2 m[8];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int c = lane - (16 * half + j);
                    float e = fmaf(__uint_as_float(v[j]), f[j], c == 0 ? Dh : 0.f);  // D x_t
                    e = c >= 0 ? e : 0.f;
                    if (j & 1)
                        m[j / 2].y = e;
                    else
                        m[j / 2].x = e;
                }
                put_m(q, m);
            }
#pragma unroll 1
            for (int J = 0; J < 4; ++J) {
                if (J == q) continue;
                if (J > q) {  // nothing but later tokens
                    const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    const uint32_t at = 32 * J + 16 * half;
                    su_st8(tml + kTmS + at, zero);
                    su_st8(tml + kTmS + at + 8, zero);
                    su_st8(tml + kTmLo + at / 2, zero);
                    continue;
                }
                uint32_t v[16];
                su_ld16(tml + kTmS + 32 * J + 16 * half, v);
                const float4 o = s_sum[J];
                const float to = pre32 + ((J < 1 && q > 1 ? sums.y : 0.f) + (J < 2 && q > 2 ? sums.z : 0.f));
                float2 m[8];
                factors(J, su_exp2(A2 * (to + (half ? o.w : o.y + o.z + o.w))),
                        su_exp2(A2 * (to + (half ? 0.f : o.z + o.w))), m);
                su_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m[i] = mul2(m[i], make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
                put_m(J, m);
            }
            // the state's share of the outputs, scaled in place; Y is added to it
            const float fac = su_exp2(A2 * (before + pre32));
            const float2 fac2 = make_float2(fac, fac);
            if (!su_wait(bar_o, par)) timed_out = true;
            su_fence_after();
            {
                uint32_t o[2][16];
                su_ld16(tml + kTmY + 32 * half, o[0]);
                su_ld16(tml + kTmY + 32 * half + 16, o[1]);
                su_wait_ld();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 v =
                            mul2(fac2, make_float2(__uint_as_float(o[j][2 * i]), __uint_as_float(o[j][2 * i + 1])));
                        o[j][2 * i] = __float_as_uint(v.x);
                        o[j][2 * i + 1] = __float_as_uint(v.y);
                    }
                    su_st16(tml + kTmY + 32 * half + 16 * j, o[j]);
                }
            }
            su_wait_st();
        }
        // w x in three parts, 32 passes over 4 token rows, a 16-byte chunk per
        // thread and pass. With M to build, a warp has the more of it the larger
        // q, and the issuer waits on the products: the passes even that out.
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        __nv_bfloat162 z = zero;  // NaN when x has a NaN or infinity
        constexpr uint64_t kFirst = OUT ? 0x1D1914120F0B0600ull : 0x1C1814100C080400ull;  // byte w: warp w's first pass
        constexpr uint32_t kPasses = OUT ? 0x34523456u : 0x44444444u;                      // digit w: how many
        const int first = static_cast<int>((kFirst >> (8 * warp)) & 31), passes = (kPasses >> (4 * warp)) & 15;
        if (!su_wait(bar_x, par)) timed_out = true;
#pragma unroll 1
        for (int pass = first; pass < first + passes; ++pass) {
            const int s = 4 * pass + (lane >> 3);
            const uint32_t at = static_cast<uint32_t>(128 * s + 16 * ((lane & 7) ^ (s & 7)));
            uint4* xp = reinterpret_cast<uint4*>(smem + kSuX + at);
            uint4 u = *xp;
            if (t0 + s >= it.t1) *xp = u = make_uint4(0, 0, 0, 0);  // a row of the next request, or of none
            // dt sums of the groups of 8 after the token's in its 32-block, and of the 32-blocks after
            const float4 o = s_sum[pass >> 3];
            const int so = (pass >> 1) & 3;
            const float after = ((so < 1 ? o.y : 0.f) + (so < 2 ? o.z : 0.f) + (so < 3 ? o.w : 0.f)) +
                                ((pass < 8 ? sums.y : 0.f) + (pass < 16 ? sums.z : 0.f) + (pass < 24 ? sums.w : 0.f));
            const float w = s_col[s] * su_exp2(A2 * after);
            const float2 w2 = make_float2(w, w);
            const uint32_t xu[4] = {u.x, u.y, u.z, u.w};
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (OUT) z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&xu[i]), zero, z);
                split3(mul2(w2, bf2(xu[i])), hi[i], mid[i], lo[i]);
            }
            *reinterpret_cast<uint4*>(smem + kSuR + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(smem + kSuR + kSuBlk + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
            *reinterpret_cast<uint4*>(smem + kSuC1 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        su_fence_before();
        // M and the parts of w x are in place, x, C and the state's parts have been read
        const bool bad = __syncthreads_or(OUT && (__hisnan(z.x) || __hisnan(z.y)));
        if (OUT && bad) {
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                uint4* c = chunk(kSuX, 4 * half + j);
                const uint4 u = *c;
                *c = make_uint4(finite2(u.x), finite2(u.y), finite2(u.z), finite2(u.w));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
        }
        su_fence_after();
        if (OUT) {
            if (issuer) {
                const uint64_t dX = su_desc(sb + kSuX);
                if (elect_one()) {
                    if (more) mbar_expect_tx(bar_in, in_bytes);
#pragma unroll 1
                    for (int ks = 0; ks < kSuTok / 16; ++ks) {
                        su_mma_ts<su_idesc(64, 0, 1)>(tm + kTmY, tm + kTmS + 16 * ks, dX + 128 * ks, 1);
                        su_mma_ts<su_idesc(64, 0, 1)>(tm + kTmY, tm + kTmS + 16 * ks + 8, dX + 128 * ks, 1);
                        su_mma_ts<su_idesc(64, 0, 1)>(tm + kTmY, tm + kTmLo + 8 * ks, dX + 128 * ks, 1);
                    }
                    su_commit(bar_y);
                }
                __syncwarp();
            }
        } else if (issuer) {
            if (more && elect_one()) {
                mbar_expect_tx(bar_in, in_bytes);
                load_x(t0 + kSuTok);
            }
            __syncwarp();
        }
        d = dn;
        if (more) scan_dt();
        if (OUT) {
            if (!su_wait(bar_y, par)) timed_out = true;  // Y done, M and x read
            su_fence_after();
        }
        if (OUT && bad) {  // what was left out of Y, 8 columns at a time, before U takes M's place
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
                for (int s = 0; s < kSuTok; ++s) {
                    uint32_t hi, mid, lo;
                    su_ld1(tml + kTmS + 16 * (s >> 4) + ((s & 15) >> 1), hi);
                    su_ld1(tml + kTmS + 16 * (s >> 4) + 8 + ((s & 15) >> 1), mid);
                    su_ld1(tml + kTmLo + (s >> 1), lo);
                    su_wait_ld();
                    const float m = s & 1 ? bf_hi(hi) + (bf_hi(mid) + bf_hi(lo)) : bf_lo(hi) + (bf_lo(mid) + bf_lo(lo));
                    const uint4 u = x_given(s, 4 * half + j);
                    const uint32_t xu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t out = finite2(xu[c]) ^ xu[c];
                        if (s <= row && (out & 0xFFFFu)) acc[2 * c] = fmaf(m, bf_lo(xu[c]), acc[2 * c]);
                        if (s <= row && (out >> 16)) acc[2 * c + 1] = fmaf(m, bf_hi(xu[c]), acc[2 * c + 1]);
                    }
                }
                uint32_t y[8];
                su_ld8(tml + kTmY + 32 * half + 8 * j, y);
                su_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) + acc[i]);
                su_st8(tml + kTmY + 32 * half + 8 * j, y);
            }
            su_wait_st();
            su_fence_before();
            __syncthreads();
            su_fence_after();
        }
        if (issuer) {
            const uint64_t dB = su_desc(sb + kSuB), dR = su_desc(sb + kSuR);
            if (elect_one()) {
#pragma unroll 1
                for (int ks = 0; ks < kSuTok / 16; ++ks)
                    su_mma<su_idesc(192, 1, 1)>(tm + kTmS, dB + 128 * ks, dR + 128 * ks, ks > 0);
                su_commit(bar_u);
            }
            __syncwarp();
        }
        // Y leaves, 32 columns by way of x's buffer and 32 by way of C's first block's
        auto half_sync = [&]() {  // the four warps of this half
            if (half == 0)
                asm volatile("bar.sync 1, 128;" ::: "memory");
            else
                asm volatile("bar.sync 2, 128;" ::: "memory");
        };
        if (OUT) {
            const uint32_t stage = half == 0 ? kSuX : kSuC0;
            uint32_t y[2][16];
            su_ld16(tml + kTmY + 32 * half, y[0]);
            su_ld16(tml + kTmY + 32 * half + 16, y[1]);
            su_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t* v = &y[i >> 2][4 * (i & 3)];
                *chunk(stage, i) = make_uint4(v[0], v[1], v[2], v[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            half_sync();
            if (t0 + kSuTok <= it.t1) {
                if (warp == 0 || warp == kSuStorer) {
                    if (elect_one()) {
                        if (pb < P) su_tma_store(my, sb + stage, pb, h, t0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        if (warp == 0)  // x's buffer is free
                            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar_f) : "memory");
                        else if (more)
                            load_c0(t0 + kSuTok);
                    }
                    __syncwarp();
                }
            } else {  // not the rows of the next request: row by row
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int r = 16 * i + 4 * q + (lane >> 3), j = lane & 7;
                    const uint4 v = *reinterpret_cast<const uint4*>(smem + stage + r * 128 + 16 * (j ^ (r & 7)));
                    if (t0 + r < it.t1 && pb + 4 * j < P)
                        *reinterpret_cast<uint4*>(a.y + (static_cast<size_t>(t0 + r) * H + h) * P + pb + 4 * j) = v;
                }
            }
        }
        if (!su_wait(bar_u, par)) timed_out = true;
        su_fence_after();
        if (issuer) {
            if (more && elect_one()) load_bc(t0 + kSuTok);  // U has read B and the parts of w x
            __syncwarp();
        }
        const float dec = su_exp2(A2 * total);
        const float2 dec2 = make_float2(dec, dec);
        dtsum += total;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t u0[16], u1[16], u2[16];
            su_ld16(tml + kTmS + 32 * half + 16 * j, u0);
            su_ld16(tml + kTmS + 64 + 32 * half + 16 * j, u1);
            su_ld16(tml + kTmS + 128 + 32 * half + 16 * j, u2);
            su_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                auto two = [&](const uint32_t (&u)[16]) {
                    return make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                };
                hst[8 * j + i] = fma2(dec2, hst[8 * j + i], add2(two(u0), add2(two(u1), two(u2))));
            }
        }
        if (OUT && more) {
            if (!su_wait(bar_f, par)) timed_out = true;
            put_state();
        }
    }
    if (timed_out) set_error(a.err, RSSM_DEVERR_TIMEOUT);
    if ((!OUT || it.last) && row < N) {
        float* out = (OUT ? head_state(a, it.b, h) : slot_state(a, it.slot, h)) + static_cast<size_t>(pb) * N + row;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (pb + 2 * j < P) out[2 * j * N] = hst[j].x;
            if (pb + 2 * j + 1 < P) out[(2 * j + 1) * N] = hst[j].y;
        }
    }
    if (!OUT && tid == 0 && p0 == 0) *slot_dtsum(a, it.slot, h) = dtsum;
    su_fence_before();
    __syncthreads();
    if (warp == 0) {
        su_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kSuCols) : "memory");
    }
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

// The tensor-core scan moves 16 bytes of an x row at a time.
bool scan_umma_shape(const Shape& s, int in_bf16) {
    return in_bf16 && s.P % 8 == 0 && static_cast<long long>(s.batch) * s.H * ((s.P + 63) / 64) <= 0x7fffffffLL;
}

// The driver's tensor-map encoder (the library links the runtime only).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static std::atomic<void*> fn{nullptr};
    void* p = fn.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

// Per-token rows [total][width] bf16, read in boxes of 128 tokens x 64
// columns (128-byte rows, swizzled); zeros outside.
bool encode_rows(CUtensorMap* m, const void* base, int total, long long width) {
    EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(total)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * width)};
    const cuuint32_t box[2] = {64, kSuTok}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [total][H][P] fp32, written in boxes of 128 tokens x 32 columns of a head.
bool encode_out(CUtensorMap* m, float* base, int total, int H, int P) {
    EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(P), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(total)};
    const cuuint64_t strides[2] = {4ull * P, 4ull * P * H};
    const cuuint32_t box[3] = {32, 1, kSuTok}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool OUT>
cudaError_t launch_umma(const ScanArgs& a, int items, cudaStream_t st) {
    const int slices = (a.s.P + 63) / 64;
    CUtensorMap mx, mb, mc, my;
    const long long xw = static_cast<long long>(a.s.H) * a.s.P, bw = static_cast<long long>(a.s.G) * a.s.N;
    if (!encode_rows(&mx, a.x, a.total, xw) || !encode_rows(&mb, a.B, a.total, bw) ||
        !encode_rows(&mc, a.C, a.total, bw) || !encode_out(&my, a.y, a.total, a.s.H, a.s.P))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(k_scan_umma<OUT>, kSuSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(items) * static_cast<unsigned>(a.s.H) * static_cast<unsigned>(slices));
    k_scan_umma<OUT><<<grid, kSuThreads, kSuSmem, st>>>(a, mx, mb, mc, my, slices);
    return cudaGetLastError();
}

// Shared memory of k_scan: two buffers of tokens and their outputs. The most
// that a supported shape takes is at head_dim 256, d_state 64 (65792 bytes).
constexpr size_t scan_smem(int P, int N) {
    return 4u * kScanTok * (2 * (2 + ((P + 3) & ~3) + 2 * static_cast<size_t>(N)) + P);
}
constexpr size_t kScanSmemMax = scan_smem(256, 64);
static_assert(scan_smem(128, 128) <= kScanSmemMax, "head_dim * d_state is at most 16384");

template <typename TIn, bool OUT>
cudaError_t launch_pass(const ScanArgs& a, int items, cudaStream_t st) {
    if (scan_umma_shape(a.s, sizeof(TIn) == 2)) return launch_umma<OUT>(a, items, st);
    const size_t smem = scan_smem(a.s.P, a.s.N);
    const int passes = (a.s.P * a.s.lpr + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(items) * static_cast<unsigned>(a.s.H));
    // the limit of every shape at once: another thread's launch of another shape must not lower it
    static std::atomic<uint64_t> allowed[5];
    auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
        const cudaError_t e = allow_smem(kernel, kScanSmemMax, done);
        if (e != cudaSuccess) return e;
        kernel<<<grid, kThreads, smem, st>>>(a);
        return cudaGetLastError();
    };
    if (passes <= 1) return go(k_scan<TIn, 1, OUT>, allowed[0]);
    if (passes <= 2) return go(k_scan<TIn, 2, OUT>, allowed[1]);
    if (passes <= 4) return go(k_scan<TIn, 4, OUT>, allowed[2]);
    if (passes <= 8) return go(k_scan<TIn, 8, OUT>, allowed[3]);
    return go(k_scan<TIn, 16, OUT>, allowed[4]);
}

}  // namespace

// Whole requests or segments, and which: the least of the times that a simple
// model of the two kernels gives. A CTA takes `alone` per step while it has an
// SM to itself and `shared` while it shares one (us per 128 tokens; measured
// on B200 at head_dim 64, d_state 128) and 5 us to start and end, the pass over
// the segments' states less; two more launches cost 15 us and the join its
// bytes. 148 SMs: the
// workspace must not depend on the device that asks. Measured against whole
// requests: one prompt of 8192 tokens, 64 heads, 350 -> 189 us in 4 segments;
// 16 prompts of up to 1501 tokens, 64 heads, 117 us whole and 148 us at best
// in segments; one of 16384 tokens, 128 heads, which the model leaves whole,
// 696 us and 647 us in 2 segments.
int scan_segment_len(const Shape& s, int in_bf16, int total, int max_seqlen) {
    struct Cost {
        int per_sm, tok;      // CTAs that share an SM; tokens per step
        double alone, shared, state_alone, state_shared;
    };
    const bool umma = scan_umma_shape(s, in_bf16);
    const Cost c = umma ? Cost{2, 128, 5.4, 8.1, 2.6, 3.8} : Cost{4, 128, 45, 150, 27, 80};
    const double heads = static_cast<double>(s.H) * (umma ? (s.P + 63) / 64 : 1);
    const long long longest = max_seqlen < total ? max_seqlen : total;
    const long long steps = (longest + c.tok - 1) / c.tok;
    auto rounds = [&](double ctas, double alone, double shared) {  // of CTAs that run at once, in us per step
        if (ctas <= 148) return alone;
        const double fit = 148.0 * c.per_sm;
        return shared * static_cast<double>(static_cast<long long>((ctas + fit - 1) / fit));
    };
    const double ctas = heads * s.batch;
    const double even = heads * (total + 0.5 * c.tok * s.batch) / c.tok / (148.0 * c.per_sm) * c.shared;
    double best = steps * (ctas <= 148 ? c.alone : c.shared);
    if (even > best) best = even;
    best *= 0.95;
    long long len = 0;
    for (long long n = 2, before = 0; n <= 64 && n <= steps; ++n) {
        const long long each = (steps + n - 1) / n, tokens = each * c.tok;
        if (each == before) continue;
        before = each;
        const double segs = static_cast<double>((total + tokens - 1) / tokens) + 0.5 * (s.batch - 1);
        const double inner = segs - s.batch > 0 ? segs - s.batch : 0;
        const double join = s.H * (segs + s.batch) * s.P * s.N * 12 / 5e6;  // us
        const double t = each * (rounds(heads * segs, c.alone, c.shared) +
                                 (inner > 0 ? rounds(heads * inner, c.state_alone, c.state_shared) : 0)) +
                         rounds(heads * segs, 5, 5) + (inner > 0 ? rounds(heads * inner, 5, 5) : 0) + 15 + join;
        // one CTA per slot and head
        if (t < best && (total / tokens + s.batch) * static_cast<long long>(heads) <= 0x7fffffffLL) {
            best = t;
            len = tokens;
        }
    }
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
