// Causal attention of ragged query blocks over a paged cache in bf16 or e4m3
// ([EN] §2.3 Eq. 2, §3.3 Algorithm 2).
//
// One CTA per (16 query rows of a kv head, sequence): a row is (query token,
// query head of the group).  Keys pass through shared memory in fp32, 32 at a
// time; a warp owns two rows, its lanes hold a score each and four output
// elements each, with the running maximum and sum of the softmax.
#include "masw_paged_attn.cuh"

#include <algorithm>
#include <cstring>

namespace masw {

constexpr int kSimpleRows = 16, kSimpleKeys = 32;

__global__ void __launch_bounds__(256) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    extern __shared__ float fs[];
    const PagedView& c = p.c;
    const int D = c.D, LD = D + 1;
    float* qs = fs;                              // [16][D]
    float* ks = qs + kSimpleRows * D;            // [32][D + 1]
    float* vs = ks + kSimpleKeys * LD;           // [32][D + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, h = blockIdx.y, G = p.G;
    const SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, c.B, c.cap);
    const bool bad = !s.ok || s.n > p.max_rows;
    if (bad && tid == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
    if (bad) return;
    const int n0 = (int)blockIdx.x * kSimpleRows, n1 = imin(s.n * G, n0 + kSimpleRows);
    if (n0 >= n1) return;
    for (int i = tid; i < kSimpleRows * D; i += blockDim.x) {
        const int n = n0 + i / D;
        qs[i] = n < n1 ? __bfloat162float(p.q[(size_t)(s.r0 + n / G) * p.q_stride + (size_t)(h * G + n % G) * D + i % D]) : 0.f;
    }
    const int p_first = s.kv - s.n + n0 / G, p_last = s.kv - s.n + (n1 - 1) / G;   // positions of the rows
    const int k_end = imax(0, imin(s.kv, p_last + 1));
    const int k_beg = p.window > 0 ? imax(0, p_first - p.window + 1) : 0;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][4] = {};
    for (int k0 = k_beg; k0 < k_end; k0 += kSimpleKeys) {
        __syncthreads();
        for (int i = tid; i < kSimpleKeys * D; i += blockDim.x) {
            const int kk = k0 + i / D, d = i % D;
            float kx = 0.f, vx = 0.f;
            if (kk < k_end) {
                const int pid = c.table[(size_t)b * c.table_stride + kk / c.P];
                if (pid < 0 || pid >= c.n_pages) {
                    if (p.status) atomicExch(p.status, MASW_EINVAL);
                } else {
                    const size_t at = ((size_t)h * c.P + kk % c.P) * D + d, page = (size_t)pid * c.page_bytes;
                    if (c.k_scale) {
                        float hi;
                        f16x2_to_f32(e4m3x2_to_f16x2(c.k[page + at]), kx, hi);
                        f16x2_to_f32(e4m3x2_to_f16x2(c.v[page + at]), vx, hi);
                        kx *= c.k_scale[(size_t)pid * c.Hkv + h];
                        vx *= c.v_scale[(size_t)pid * c.Hkv + h];
                    } else {
                        kx = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(c.k + page)[at]);
                        vx = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(c.v + page)[at]);
                    }
                }
            }
            ks[(i / D) * LD + d] = kx;
            vs[(i / D) * LD + d] = vx;
        }
        __syncthreads();
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            const int n = n0 + warp * 2 + rr;
            if (n >= n1) continue;
            const int pos = s.kv - s.n + n / G, key = k0 + lane;
            const bool see = key < k_end && key <= pos && (p.window <= 0 || key > pos - p.window);
            float x = 0.f;
            for (int d = 0; d < D; ++d) x = fmaf(qs[(n - n0) * D + d], ks[lane * LD + d], x);
            x = see ? x * p.scale : -INFINITY;
            float mx = x;
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m[rr], mx);
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float a = expf(m[rr] - ref), pr = see ? expf(x - ref) : 0.f;
            float sum = pr;
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[rr] = l[rr] * a + sum;
            m[rr] = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[rr][e] *= a;
            for (int kk = 0; kk < kSimpleKeys; ++kk) {
                const float w = __shfl_sync(0xffffffffu, pr, kk);
                if (w == 0.f) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (lane + 32 * e < D) acc[rr][e] = fmaf(w, vs[kk * LD + lane + 32 * e], acc[rr][e]);
            }
        }
    }
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
        const int n = n0 + warp * 2 + rr;
        if (n >= n1) continue;
        const size_t row = (size_t)(s.r0 + n / G) * p.Hq + (size_t)h * G + n % G;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = lane + 32 * e;
            if (d >= D) continue;
            const float x = l[rr] == 0.f ? 0.f : acc[rr][e] / l[rr];
            if (p.o_f32) ((float*)p.o)[row * D + d] = x;
            else ((__nv_bfloat16*)p.o)[row * D + d] = __float2bfloat16_rn(x);
        }
        if (lane == 0 && p.lse) p.lse[row] = l[rr] == 0.f ? -INFINITY : m[rr] + logf(l[rr]);
    }
}

}  // namespace masw

using namespace masw;

static int paged_attn_sizes(const PagedView& c, const char* who, int rows, int max_rows, bool ragged, int n_q_heads, int* mr) {
    auto fail = [&](const char* why) { return masw_set_error(nullptr, MASW_EINVAL, std::string(who) + ": " + why); };
    if (rows < 0) return fail("rows must not be negative");
    if (!ragged && rows % c.B) return fail("without row_start, rows must be a multiple of batch");
    if (ragged && max_rows < 0) return fail("max_rows must not be negative");
    if (n_q_heads < c.Hkv || n_q_heads % c.Hkv || n_q_heads / c.Hkv > 128)
        return fail("n_q_heads must be a multiple of n_kv_heads, at most 128 per kv head");
    if ((long long)rows * n_q_heads > 0x7fffffffll) return fail("rows * n_q_heads must be below 2^31");
    *mr = ragged ? std::min(max_rows, rows) : rows / c.B;
    if ((long long)c.B * c.Hkv * (c.cap / kTile + 2) > 0x7fffffffll) return fail("batch * heads * table too large");
    return MASW_OK;
}

static int device_sms(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return masw_set_error(nullptr, MASW_ECUDA, "paged_attn: cannot query the current device");
    }
    return MASW_OK;
}

static size_t workspace_bytes_for(const PagedView& c, int max_rows, int G, int sms) {
    if ((long long)max_rows * G > kRowsMax) return 16;
    return (size_t)sms * 2 * kRowsMax * (c.D + 2) * sizeof(float);   // two partials a CTA
}

// pages as a 4-d tensor [n_pages][Hkv][P][D], boxes of one page's rows (at most
// 128) and one 128-byte (or narrower) column panel, swizzled as the matrix
// descriptors say
static bool make_page_map(CUtensorMap* map, const PagedView& c, const uint8_t* base) {
    const int esize = c.k_scale ? 1 : 2, row = c.D * esize, panel = std::min(row, 128);
    const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.P, (cuuint64_t)c.Hkv, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)row, (cuuint64_t)c.P * row, (cuuint64_t)c.page_bytes};
    const cuuint32_t box[4] = {(cuuint32_t)(panel / esize), (cuuint32_t)std::min(c.P, kTile), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return tma_encode_fn()(map, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<uint8_t*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           panel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" int masw_paged_workspace_bytes(const masw_paged_t* cache, int rows, int max_rows, int n_q_heads, size_t* bytes) {
    if (!bytes) return masw_set_error(nullptr, MASW_EINVAL, "paged_workspace: bytes is NULL");
    PagedView c;
    int rc = masw_paged_view(cache, "paged_workspace", &c);
    int mr = 0;
    if (!rc) rc = paged_attn_sizes(c, "paged_workspace", rows, max_rows, true, n_q_heads, &mr);
    if (rc) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    *bytes = workspace_bytes_for(c, mr, n_q_heads / c.Hkv, sms);
    return MASW_OK;
}

extern "C" int masw_paged_attn(const masw_paged_t* cache, const int* kv_len, const int* row_start, int rows, int max_rows,
                               const void* q, int n_q_heads, long long q_stride, int window, float scale, void* o,
                               int o_dtype, float* lse, int* status, void* workspace, size_t workspace_bytes,
                               masw_stream_t stream) {
    PagedAttnParams p;
    std::memset(&p, 0, sizeof(p));
    int mr = 0;
    int rc = masw_paged_view(cache, "paged_attn", &p.c);
    if (!rc) rc = paged_attn_sizes(p.c, "paged_attn", rows, max_rows, row_start != nullptr, n_q_heads, &mr);
    if (rc) return rc;
    auto fail = [&](const char* why) { return masw_set_error(nullptr, MASW_EINVAL, std::string("paged_attn: ") + why); };
    if (!kv_len || !q || !o || !workspace) return fail("NULL pointer");
    if (o_dtype != MASW_BF16 && o_dtype != MASW_F32) return fail("o_dtype must be MASW_BF16 or MASW_F32");
    if (window < 0) return fail("window must not be negative");
    if (!(scale >= 0.f && scale <= 3.0e38f)) return fail("scale must be finite and not negative");
    const long long qd = (long long)n_q_heads * p.c.D;
    p.q_stride = q_stride ? q_stride : qd;
    if (p.q_stride < qd || p.q_stride & 7) return fail("q_stride must hold a token's heads and be a multiple of 8");
    if (((uintptr_t)q | (uintptr_t)o | (uintptr_t)workspace) & 15) return fail("q, o and workspace must be 16-byte aligned");
    if (((uintptr_t)kv_len | (uintptr_t)row_start | (uintptr_t)lse | (uintptr_t)status) & 3)
        return fail("kv_len, row_start, lse and status must be 4-byte aligned");
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    if (workspace_bytes < workspace_bytes_for(p.c, mr, n_q_heads / p.c.Hkv, sms)) return fail("workspace too small");
    if (rows == 0 || mr == 0) return MASW_OK;
    if (!tma_encode_fn()) return masw_set_error(nullptr, MASW_ECUDA, "paged_attn: cuTensorMapEncodeTiled is unavailable");
    if (!make_page_map(&p.tm_k, p.c, p.c.k) || !make_page_map(&p.tm_v, p.c, p.c.v))
        return fail("cannot describe the pages as TMA tensors");
    p.part = (float*)workspace;
    p.kv_len = kv_len;
    p.row_start = row_start;
    p.q = (const __nv_bfloat16*)q;
    p.o = o;
    p.lse = lse;
    p.status = status;
    p.rows = rows;
    p.max_rows = mr;
    p.Hq = n_q_heads;
    p.G = n_q_heads / p.c.Hkv;
    p.window = window;
    p.o_f32 = o_dtype == MASW_F32;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)p.c.D);
    p.scale_log2 = p.scale * 1.4426950408889634f;
    if (mr * p.G <= kRowsMax) {
        const cudaError_t e = launch_paged_rows(p, sms, (cudaStream_t)stream);
        if (e != cudaSuccess) return masw_set_error(nullptr, MASW_ECUDA, std::string("paged_attn: ") + cudaGetErrorString(e));
        return MASW_OK;
    }
    const size_t smem = (size_t)(kSimpleRows * p.c.D + 2 * kSimpleKeys * (p.c.D + 1)) * sizeof(float);
    const long long tiles = ((long long)mr * p.G + kSimpleRows - 1) / kSimpleRows;
    const cudaError_t e = masw_launch(paged_attn_kernel, dim3((unsigned)tiles, p.c.Hkv, p.c.B), dim3(256), smem,
                                      (cudaStream_t)stream, 1, p);
    if (e != cudaSuccess) return masw_set_error(nullptr, MASW_ECUDA, std::string("paged_attn: ") + cudaGetErrorString(e));
    return MASW_OK;
}
