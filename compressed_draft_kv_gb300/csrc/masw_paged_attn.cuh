// Parameters and device helpers shared by the paged attention kernels.
#pragma once

#include "masw_paged.cuh"
#include "masw_tc.cuh"

#include <atomic>
#include <type_traits>

namespace masw {

constexpr int kRowsMax = 32;   // query rows of a pair that the few-rows kernel takes

struct PagedAttnParams {
    CUtensorMap tm_k;         // pages as [n_pages][Hkv][P][D], boxes of one page's rows (at most 128)
    CUtensorMap tm_v;
    PagedView c;
    const int* kv_len;
    const int* row_start;
    const __nv_bfloat16* q;   // [rows][Hq][D], token stride q_stride
    long long q_stride;
    void* o;
    float* lse;
    int* status;
    float* part;              // partial results of pairs cut over CTAs
    int rows, max_rows, Hq, G, window, o_f32;
    float scale, scale_log2;
};

__device__ __forceinline__ void store_out(const PagedAttnParams& p, size_t at, float x) {
    if (p.o_f32) reinterpret_cast<float*>(p.o)[at] = x;
    else reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(x);
}

// The line of all pairs' tiles: pre[b] = tiles before sequence b, pre[B] = all
// of them (returned), and the sequences' rows and lengths, by the whole CTA of NT
// threads.  A sequence whose rows or length are not possible has no tiles.
template <int NT>
__device__ int make_line(const PagedAttnParams& p, int* pre, int* s_kv, int* s_n, int* s_r0, bool report) {
    constexpr int kPer = (MASW_MAX_BATCH + NT - 1) / NT;
    __shared__ int warp_sum[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, B = p.c.B;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int b = tid * kPer + k;
        mine[k] = 0;
        if (b < B) {
            SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, B, p.c.cap);
            if (!s.ok || s.n > p.max_rows) {
                if (report && p.status) atomicExch(p.status, MASW_EINVAL);
                s.n = s.kv = 0;
            }
            s_kv[b] = s.kv;
            s_n[b] = s.n;
            s_r0[b] = s.r0;
            mine[k] = tile_range(s.n, s.kv, p.window).nt * p.c.Hkv;
        }
        sum += mine[k];
    }
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
    }
    if (lane == 31) warp_sum[tid >> 5] = scan;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < tid >> 5) before += warp_sum[w];
        total += warp_sum[w];
    }
    before += scan - sum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int b = tid * kPer + k;
        if (b < B) pre[b] = before;
        before += mine[k];
    }
    if (tid == 0) pre[B] = total;
    __syncthreads();
    return total;
}

// The few-rows kernel and its merge on n_cta CTAs (masw_paged_rows.cu).
cudaError_t launch_paged_rows(const PagedAttnParams& p, int n_cta, cudaStream_t st);

}  // namespace masw
