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
    CUtensorMap tm_q;         // many rows: Q as [rows][Hq][D], boxes of a tile's tokens and one kv head's heads
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

// A bounded wait in few instructions and registers (the kernels are large, and what
// stalled them most was fetching instructions): barrier and abort flag by their
// shared-memory addresses.  try_wait itself suspends the thread for a while.  One
// wait that gives up sets the flag, and every later one returns at once.
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t at, uint32_t v) {
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint32_t abort_flag, int* status) {
    uint32_t n = 0;
#pragma unroll 1
    while (!mbar_try_wait_at(bar, parity)) {
        if (ld_shared_u32(abort_flag)) return false;
        if (++n == kWaitPolls) {
            st_shared_u32(abort_flag, 1u);
            if (status) atomicExch(status, MASW_ETIMEOUT);
            return false;
        }
    }
    return true;
}

// N consecutive fp32 columns (a multiple of 8) of this thread's TMEM lane
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* v) {
    if constexpr (N >= 32) {
        tc::tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld_cols<N - 32>(taddr + 32, v + 32);
    } else if constexpr (N >= 16) {
        tc::tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(v));
        tmem_ld_cols<N - 16>(taddr + 16, v + 16);
    } else if constexpr (N >= 8) {
        tc::tmem_ld8(taddr, *reinterpret_cast<uint32_t(*)[8]>(v));
    }
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// two f16 pairs -> four e4m3, rounded to nearest
__device__ __forceinline__ uint32_t e4m3x4(uint32_t h0, uint32_t h1) {
    uint32_t r;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}\n"
        : "=r"(r)
        : "r"(h0), "r"(h1));
    return r;
}
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t v, uint32_t& h0, uint32_t& h1) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(h0), "=r"(h1)
        : "r"(v));
}
// The line of all pairs' tiles: pre[b] = tiles before sequence b, pre[B] = all
// of them, and the sequences' rows and lengths, by the whole CTA of NT
// threads.  A sequence whose rows or length are not possible has no tiles.
struct Line {
    int total, longest;      // tiles of all pairs, and of the longest
};
template <int NT>
__device__ Line make_line(const PagedAttnParams& p, int* pre, int* s_kv, int* s_n, int* s_r0, bool report) {
    constexpr int kPer = (MASW_MAX_BATCH + NT - 1) / NT;
    __shared__ int warp_sum[NT / 32], warp_top[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, B = p.c.B;
    int mine[kPer], sum = 0, top = 0;
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
            const int nt = tile_range(s.n, s.kv, p.window).nt;
            mine[k] = nt * p.c.Hkv;
            top = imax(top, nt);
        }
        sum += mine[k];
    }
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 31) {
        warp_sum[tid >> 5] = scan;
        warp_top[tid >> 5] = top;
    }
    __syncthreads();
    int before = 0, total = 0, longest = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < tid >> 5) before += warp_sum[w];
        total += warp_sum[w];
        longest = imax(longest, warp_top[w]);
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
    return Line{total, longest};
}

// How the many-rows kernel cuts its work: `items` of 256 rows a (sequence, kv head)
// pair, in the order of unit_of; the first `whole` units take a CTA each and the last
// `cut` n_split CTAs, along the keys if they have at least min_tiles tiles of them.
struct TilePlan {
    int items, group, whole, cut, n_split, min_tiles;
};
// The many-rows kernel and its merge (masw_paged_tile.cu).
cudaError_t launch_paged_tiles(const PagedAttnParams& p, const TilePlan& plan, cudaStream_t st);

// The few-rows kernel and its merge on n_cta CTAs (masw_paged_rows.cu).
cudaError_t launch_paged_rows(const PagedAttnParams& p, int n_cta, cudaStream_t st);

}  // namespace masw
