// Causal attention of ragged query blocks over a paged cache in bf16 or e4m3
// ([EN] §2.3 Eq. 2, §3.3 Algorithm 2).
//
// Two kernels, by the number of query rows (query token x query head of the
// group) of a (sequence, kv head) pair: up to 32 go to the few-rows kernel
// (masw_paged_rows.cu: keys as the matrix rows, bound by reading the cache), more
// to the many-rows kernel (masw_paged_tile.cu: query rows as the matrix rows).
#include "masw_paged_attn.cuh"

#include <algorithm>
#include <cstring>

namespace masw {

// The plan of the many-rows kernel: 128 / G tokens a tile, two tiles an item, one
// CTA an SM.  Fewer items than SMs: all are cut into as many splits as fill the SMs
// once.  A few waves of items: those of the last, partly filled wave are cut so that
// it ends sooner (256 items on 152 SMs: 104 of them in 7 parts each, 1.7 waves
// instead of 2), if they have 8K keys at least: a 4K chunk at 16K takes 706 us so
// and 744 uncut, but a 4K prompt, whose last items are short, 134 us and 115 uncut.
// Many waves: nothing is cut, the end of the last one costs little.
static TilePlan tile_plan(const PagedView& c, int max_rows, int G, int sms) {
    TilePlan t;
    const int tokens = 2 * (kTile / G);
    t.items = (max_rows + tokens - 1) / tokens;
    const long long units = (long long)t.items * c.Hkv * c.B;
    const long long pairs = (long long)c.B * c.Hkv, groups = std::min(pairs, std::max(1ll, units / (6ll * sms)));
    t.group = (int)((pairs + groups - 1) / groups);
    t.cut = 0;
    t.min_tiles = 0;
    t.n_split = 1;
    if (units < sms) {
        t.n_split = (int)std::min<long long>(64, sms / units);
        t.cut = t.n_split > 1 ? (int)units : 0;
    } else if (units < 6ll * sms) {
        const int rest = (int)(units % sms);
        double best = 0.9;
        t.min_tiles = 64;
        for (int n = 2; n <= 8; ++n) {
            const double waves = (double)(((long long)rest * n + sms - 1) / sms) / n;
            if (rest && waves < best - 0.01) {
                best = waves;
                t.n_split = n;
                t.cut = rest;
            }
        }
    }
    t.whole = (int)(units - t.cut);
    return t;
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
    if (((long long)rows * (n_q_heads / c.Hkv) / 128 + 1) * c.Hkv * c.B > 0x3fffffffll) return fail("too many rows and heads");
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
    if ((long long)max_rows * G > kRowsMax) {
        const TilePlan t = tile_plan(c, max_rows, G, sms);
        return t.cut == 0 ? 16 : (size_t)t.cut * t.n_split * 256 * (c.D + 2) * sizeof(float);
    }
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

// Q [rows][Hq][D] (token stride q_stride), boxes of 128 / G tokens x G heads x 64
// elements, swizzled
static bool make_q_map(CUtensorMap* map, const PagedAttnParams& p) {
    const cuuint64_t dims[3] = {(cuuint64_t)p.c.D, (cuuint64_t)p.Hq, (cuuint64_t)p.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)p.c.D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(kTile / p.G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return tma_encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    if (workspace_bytes < 16) return fail("workspace too small");
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
    cudaError_t e;
    if ((long long)mr * p.G <= kRowsMax) {
        e = launch_paged_rows(p, sms, (cudaStream_t)stream);
    } else {
        const TilePlan t = tile_plan(p.c, mr, p.G, sms);
        if (p.q_stride >= (1ll << 39) || !make_q_map(&p.tm_q, p)) return fail("cannot describe q as a TMA tensor");
        e = launch_paged_tiles(p, t, (cudaStream_t)stream);
    }
    if (e != cudaSuccess) return masw_set_error(nullptr, MASW_ECUDA, std::string("paged_attn: ") + cudaGetErrorString(e));
    return MASW_OK;
}
