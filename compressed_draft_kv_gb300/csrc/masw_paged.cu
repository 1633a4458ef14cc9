// Append to a paged K/V cache ([EN] §3.3 Algorithm 2: the verified block's keys
// and values join the target's cache) with the rotary rotation of K and Q on the
// way, and the argument checks of the paged-cache calls.
//
// One CTA works on one (sequence, touched page) unit and up to 256 / (D / 16)
// heads of K, V and Q.  D / 16 lanes own one head: they walk the page's new rows
// twice, first for the largest magnitude (e4m3 pages: the page's scale must
// cover them all before one is stored), then to store.  A (page, head) belongs
// to one group of lanes, so its scale needs no atomics and the result does not
// depend on timing.  Bound by HBM for prompts (bf16 rows in, pages out), by the
// chain of dependent loads (row range, length, page id, old scale, rows) for a
// decode step.
#include "masw_paged.cuh"

#include <algorithm>
#include <cstring>

namespace masw {

struct PagedAppendParams {
    PagedView c;
    const int* kv_len;
    const int* row_start;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const __nv_bfloat16* q;
    __nv_bfloat16* q_out;
    long long k_stride, v_stride, q_stride;   // elements between token rows
    const float* cos_sin;
    const int* pos;
    int n_pos, rot, interleaved;
    int rows, Hq;
    int* status;
};

// Sixteen elements of a head held by one lane: two chunks of eight.  Lane t of
// the D / 16 lanes of a head holds, within the rotated part, the chunks whose
// elements pair up (the t-th eight of each half, or sixteen consecutive ones
// when pairs are adjacent); behind it sixteen consecutive elements.
struct LaneChunks {
    int c0, c1;      // first element of each chunk
    int ang;         // first angle index, or -1: not rotated
};
__host__ __device__ inline LaneChunks lane_chunks(int t, int rot, int interleaved) {
    if (16 * t >= rot) return LaneChunks{16 * t, 16 * t + 8, -1};
    if (interleaved) return LaneChunks{16 * t, 16 * t + 8, 8 * t};
    return LaneChunks{8 * t, rot / 2 + 8 * t, 8 * t};
}

__device__ __forceinline__ void load_rotated(const __nv_bfloat16* src, const LaneChunks& lc, bool rotate, const float* cs,
                                             int rot, int interleaved, float (&x)[16]) {
    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(src + lc.c0), x);
    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(src + lc.c1), x + 8);
    if (!rotate || lc.ang < 0) return;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + lc.ang + i);
        *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + rot / 2 + lc.ang + i);
    }
    // each product and sum rounded once (no fused multiply-add), so the stored
    // values are those of the written formula
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = x[i + 8];
            x[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            x[i + 8] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
    }
}

__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const LaneChunks& lc, const float (&x)[16]) {
    *reinterpret_cast<uint4*>(dst + lc.c0) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    *reinterpret_cast<uint4*>(dst + lc.c1) =
        make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
}

// the sequence of unit `u`: the last one whose first unit is not behind it
__device__ int find_sequence(const PagedAppendParams& p, int u) {
    int found = 0;
    for (int i0 = 0; i0 < p.c.B; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        int r0 = 0;
        if (i < p.c.B) r0 = p.row_start ? p.row_start[i] : i * (p.rows / p.c.B);
        found += __syncthreads_count(i < p.c.B && append_unit_base(imax(0, r0), i, p.c.P) <= u);
    }
    return imax(0, found - 1);
}

__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
    pdl_wait();
    pdl_trigger();
    const PagedView& c = p.c;
    const int tid = threadIdx.x, P = c.P;
    // one CTA checks every sequence's row range and length
    if (p.status && blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = tid; i < c.B; i += blockDim.x) {
            const SeqRows s = seq_rows(p.row_start, p.kv_len, i, p.rows, c.B, c.cap);
            if (!s.ok || s.n > s.kv) atomicExch(p.status, MASW_EINVAL);
        }
    const int u = blockIdx.x, b = find_sequence(p, u);
    const SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, c.B, c.cap);
    if (s.n < 1 || s.n > s.kv) return;
    const int p0 = s.kv - s.n, lp = u - append_unit_base(s.r0, b, P);
    const int page = p0 / P + lp;
    if (lp < 0 || page > (s.kv - 1) / P) return;
    const int ra = imax(p0, page * P), rb = imin(s.kv, (page + 1) * P);   // positions of this unit's rows
    const int pid = c.table[(size_t)b * c.table_stride + page];
    const bool placed = pid >= 0 && pid < c.n_pages;
    if (!placed && tid == 0 && p.status) atomicExch(p.status, MASW_EINVAL);

    const int L = c.D / 16, t = tid % L, heads = 2 * c.Hkv + (p.q ? p.Hq : 0);
    const int hh = (int)blockIdx.y * ((int)blockDim.x / L) + tid / L;
    const bool is_q = hh >= 2 * c.Hkv, is_v = !is_q && hh >= c.Hkv;
    const bool live = hh < heads && (is_q || placed);
    const int h = is_q ? hh - 2 * c.Hkv : (is_v ? hh - c.Hkv : hh);
    const __nv_bfloat16* src = is_q ? p.q : (is_v ? p.v : p.k);
    const long long stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
    const bool rotate = p.cos_sin != nullptr && !is_v;
    const LaneChunks lc = lane_chunks(t, rotate ? p.rot : 0, p.interleaved);
    auto load = [&](int pos, float (&x)[16]) {
        const int row = s.r0 + pos - p0;
        const int rp = p.pos ? p.pos[row] : pos;
        const bool in = rp >= 0 && rp < p.n_pos;
        if (rotate && !in && t == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
        load_rotated(src + (size_t)row * stride + (size_t)h * c.D, lc, rotate && in, p.cos_sin + (size_t)(in ? rp : 0) * p.rot,
                     p.rot, p.interleaved, x);
    };
    float x[16];
    if (is_q) {
        if (live)
            for (int pos = ra; pos < rb; ++pos) {
                load(pos, x);
                store_bf16(p.q_out + ((size_t)(s.r0 + pos - p0) * p.Hq + h) * c.D, lc, x);
            }
    } else if (!c.k_scale) {
        if (live)
            for (int pos = ra; pos < rb; ++pos) {
                load(pos, x);
                uint8_t* page0 = (is_v ? c.v : c.k) + (size_t)pid * c.page_bytes;
                store_bf16(reinterpret_cast<__nv_bfloat16*>(page0) + ((size_t)h * P + pos % P) * c.D, lc, x);
            }
    }
    if (!c.k_scale) return;
    float amax = 0.f;
    if (live && !is_q)
        for (int pos = ra; pos < rb; ++pos) {
            load(pos, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[i]));
        }
    for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live || is_q) return;
    float* sp = (is_v ? c.v_scale : c.k_scale) + (size_t)pid * c.Hkv + h;
    uint8_t* base = (is_v ? c.v : c.k) + (size_t)pid * c.page_bytes + (size_t)h * P * c.D;
    const int off = ra - page * P;
    float sc = pow2_scale(amax);
    if (off > 0) {
        const float old = *sp;
        sc = amax > 0.f ? fmaxf(sc, old) : old;
        if (sc > old) {
            // rows already there are rounded again to the larger scale
            const float f = old / sc;
            for (int r = 0; r < off; ++r) {
                uint4* rp = reinterpret_cast<uint4*>(base + (size_t)r * c.D) + t;
                uint4 w = *rp;
                uint32_t* wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a0, a1, a2, a3;
                    f16x2_to_f32(e4m3x2_to_f16x2(wp[i] & 0xffffu), a0, a1);
                    f16x2_to_f32(e4m3x2_to_f16x2(wp[i] >> 16), a2, a3);
                    wp[i] = e4m3x2(a0 * f, a1 * f) | (e4m3x2(a2 * f, a3 * f) << 16);
                }
                *rp = w;
            }
        }
    }
    for (int pos = ra; pos < rb; ++pos) {
        load(pos, x);
        uint8_t* dst = base + (size_t)(pos % P) * c.D;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3x2(x[4 * i] / sc, x[4 * i + 1] / sc) | (e4m3x2(x[4 * i + 2] / sc, x[4 * i + 3] / sc) << 16);
        *reinterpret_cast<uint2*>(dst + lc.c0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + lc.c1) = make_uint2(w[2], w[3]);
    }
    if (t == 0) *sp = sc;
}

}  // namespace masw

using namespace masw;

int masw_paged_view(const masw_paged_t* cache, const char* who, PagedView* view) {
    auto fail = [&](const char* why) { return masw_set_error(nullptr, MASW_EINVAL, std::string(who) + ": " + why); };
    if (!cache) return fail("NULL cache");
    const masw_paged_t& c = *cache;
    if (c.dtype != MASW_BF16 && c.dtype != MASW_E4M3) return fail("the cache's dtype must be MASW_BF16 or MASW_E4M3");
    if (c.head_dim != 64 && c.head_dim != 128) return fail("head_dim must be 64 or 128");
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)))
        return fail("page_size must be 16, 32, 64, 128 or 256");
    if (c.batch < 1 || c.batch > MASW_MAX_BATCH) return fail("batch must be 1..512");
    if (c.n_pages < 1 || c.n_kv_heads < 1 || c.n_kv_heads > 65535 || c.table_stride < 1)
        return fail("n_pages, n_kv_heads and table_stride must be positive");
    if ((long long)c.table_stride * c.page_size > 0x7fffffffll - 256) return fail("table_stride * page_size must be below 2^31");
    if ((long long)c.batch * c.n_kv_heads * c.table_stride > (1ll << 40)) return fail("page table too large");
    if (!c.k || !c.v || !c.page_table) return fail("NULL cache pointer");
    const bool e4 = c.dtype == MASW_E4M3;
    if (e4 && (!c.k_scale || !c.v_scale)) return fail("e4m3 pages need k_scale and v_scale");
    const int esize = e4 ? 1 : 2;
    const long long dense = (long long)c.n_kv_heads * c.page_size * c.head_dim;
    const long long ps = c.page_stride ? c.page_stride : dense;
    if (ps < dense || (ps * esize) % 16) return fail("page_stride must hold a page and be a multiple of 16 bytes");
    if (ps * esize >= (1ll << 40) || ps > (1ll << 62) / c.n_pages) return fail("page_stride too large");
    if (((uintptr_t)c.k | (uintptr_t)c.v) & 15) return fail("k and v pages must be 16-byte aligned");
    if (((uintptr_t)c.page_table | (uintptr_t)c.k_scale | (uintptr_t)c.v_scale) & 3)
        return fail("page table and scales must be 4-byte aligned");
    view->k = (uint8_t*)c.k;
    view->v = (uint8_t*)c.v;
    view->k_scale = e4 ? c.k_scale : nullptr;
    view->v_scale = e4 ? c.v_scale : nullptr;
    view->table = c.page_table;
    view->page_bytes = ps * esize;
    view->n_pages = c.n_pages;
    view->P = c.page_size;
    view->Hkv = c.n_kv_heads;
    view->D = c.head_dim;
    view->B = c.batch;
    view->table_stride = c.table_stride;
    view->cap = c.table_stride * c.page_size;
    return MASW_OK;
}

extern "C" int masw_paged_append(const masw_paged_t* cache, const int* kv_len, const int* row_start, int rows,
                                 const void* k, const void* v, long long k_stride, long long v_stride,
                                 const masw_rope_t* rope, const int* pos, const void* q, void* q_out, int n_q_heads,
                                 long long q_stride, int* status, masw_stream_t stream) {
    PagedAppendParams p;
    std::memset(&p, 0, sizeof(p));
    int rc = masw_paged_view(cache, "paged_append", &p.c);
    if (rc) return rc;
    auto fail = [&](const char* why) { return masw_set_error(nullptr, MASW_EINVAL, std::string("paged_append: ") + why); };
    if (rows < 0) return fail("rows must not be negative");
    if (!row_start && rows % p.c.B) return fail("without row_start, rows must be a multiple of batch");
    if (!kv_len || !k || !v) return fail("NULL pointer");
    const long long kvd = (long long)p.c.Hkv * p.c.D;
    p.k_stride = k_stride ? k_stride : kvd;
    p.v_stride = v_stride ? v_stride : kvd;
    if (p.k_stride < kvd || p.v_stride < kvd || (p.k_stride | p.v_stride) & 7)
        return fail("k_stride and v_stride must hold a token's heads and be multiples of 8");
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out) & 15) return fail("k, v, q and q_out must be 16-byte aligned");
    if (((uintptr_t)kv_len | (uintptr_t)row_start | (uintptr_t)pos | (uintptr_t)status) & 3)
        return fail("kv_len, row_start, pos and status must be 4-byte aligned");
    if (q) {
        if (!q_out) return fail("q needs q_out");
        if (n_q_heads < 1 || n_q_heads > 65535) return fail("n_q_heads must be 1..65535");
        const long long qd = (long long)n_q_heads * p.c.D;
        p.q_stride = q_stride ? q_stride : qd;
        if (p.q_stride < qd || p.q_stride & 7) return fail("q_stride must hold a token's heads and be a multiple of 8");
        if (q == q_out && p.q_stride != qd) return fail("q_out == q needs a dense q");
        p.q = (const __nv_bfloat16*)q;
        p.q_out = (__nv_bfloat16*)q_out;
        p.Hq = n_q_heads;
    }
    if (rope) {
        if (!rope->cos_sin || rope->n_pos < 1) return fail("rope: cos_sin is NULL or empty");
        if (rope->rot_dim < 16 || rope->rot_dim > p.c.D || rope->rot_dim % 16)
            return fail("rope: rot_dim must be a multiple of 16, at most head_dim");
        if ((uintptr_t)rope->cos_sin & 15) return fail("rope: cos_sin must be 16-byte aligned");
        p.cos_sin = rope->cos_sin;
        p.n_pos = rope->n_pos;
        p.rot = rope->rot_dim;
        p.interleaved = rope->interleaved ? 1 : 0;
        p.pos = pos;
    }
    if (rows == 0) return MASW_OK;
    p.kv_len = kv_len;
    p.row_start = row_start;
    p.k = (const __nv_bfloat16*)k;
    p.v = (const __nv_bfloat16*)v;
    p.rows = rows;
    p.status = status;
    const int per_cta = 256 / (p.c.D / 16), heads = 2 * p.c.Hkv + p.Hq;
    const int gy = (heads + per_cta - 1) / per_cta;
    const cudaError_t e = masw_launch(paged_append_kernel, dim3(append_units(rows, p.c.B, p.c.P), gy), dim3(256), 0,
                                      (cudaStream_t)stream, 1, p);
    if (e != cudaSuccess) return masw_set_error(nullptr, MASW_ECUDA, std::string("paged_append: ") + cudaGetErrorString(e));
    return MASW_OK;
}
