// Append to a paged K/V cache ([EN] §3.3 Algorithm 2: the verified block's keys
// and values join the target's cache) with the rotary rotation of K and Q on the
// way, and the argument checks of the paged-cache calls.
//
// Work is cut into units of one touched page of one sequence.  A (page, head)
// belongs to one group of threads, so its scale needs no atomics and the result
// does not depend on timing.  Two kernels: in the one for steps a few lanes own
// a head and walk the unit's few rows; in the one for many rows a CTA holds all
// rows of a (page, head) at once.
#include "masw_paged.cuh"

#include <algorithm>
#include <cstring>

namespace masw {

constexpr int kStages = 3;   // heads on their way to shared memory, in the kernel for many rows, and the one at work

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
    int per_seq;   // units of every sequence, or 0: rows differ, append_unit_base
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

// The rotation of a lane's sixteen elements by o = eight cosines, eight sines:
// element i of the first chunk with element i of the second, or adjacent ones
// within each chunk (then rot0 and rot1 say whether a chunk is rotated).  Each
// product and sum is rounded once (no fused multiply-add), so the stored values
// are those of the written formula.
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&o)[16], int interleaved, bool rot0, bool rot1) {
    auto turn = [](float& a, float& b, float c, float s) {
        const float a0 = a, b0 = b;
        a = __fsub_rn(__fmul_rn(a0, c), __fmul_rn(b0, s));
        b = __fadd_rn(__fmul_rn(b0, c), __fmul_rn(a0, s));
    };
    if (interleaved) {
        if (rot0)
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], o[i], o[8 + i]);
        if (rot1)
#pragma unroll
            for (int i = 4; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], o[i], o[8 + i]);
    } else if (rot0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(x[i], x[i + 8], o[i], o[8 + i]);
    }
}

__device__ __forceinline__ void load_rotated(const __nv_bfloat16* src, const LaneChunks& lc, bool rotate, const float* cs,
                                             int rot, int interleaved, float (&x)[16]) {
    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(src + lc.c0), x);
    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(src + lc.c1), x + 8);
    if (!rotate || lc.ang < 0) return;
    float o[16];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(o + i) = *reinterpret_cast<const float4*>(cs + lc.ang + i);
        *reinterpret_cast<float4*>(o + 8 + i) = *reinterpret_cast<const float4*>(cs + rot / 2 + lc.ang + i);
    }
    rotate16(x, o, interleaved, true, true);
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
        if (i < p.c.B) r0 = p.row_start[i];
        found += __syncthreads_count(i < p.c.B && append_unit_base(imax(0, r0), i, p.c.P) <= u);
    }
    return imax(0, found - 1);
}

// one CTA checks every sequence's row range and length
__device__ __forceinline__ void check_sequences(const PagedAppendParams& p) {
    if (p.status && blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.c.B; i += blockDim.x) {
            const SeqRows s = seq_rows(p.row_start, p.kv_len, i, p.rows, p.c.B, p.c.cap);
            if (!s.ok || s.n > s.kv) atomicExch(p.status, MASW_EINVAL);
        }
}

// the page and the rows of unit `u`
struct AppendUnit {
    int ra, rb;      // positions of the unit's rows: [ra, rb)
    int row0;        // row of position 0 (row = row0 + position)
    int off;         // slots of the page before ra
    int pid;         // the page, if `placed`
    bool placed;     // the table names a page of the pool
};
__device__ __forceinline__ bool find_unit(const PagedAppendParams& p, int u, AppendUnit& w) {
    const PagedView& c = p.c;
    const int b = p.per_seq ? u / p.per_seq : find_sequence(p, u);
    const SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, c.B, c.cap);
    if (s.n < 1 || s.n > s.kv) return false;
    const int p0 = s.kv - s.n, lp = p.per_seq ? u % p.per_seq : u - append_unit_base(s.r0, b, c.P), page = p0 / c.P + lp;
    if (lp < 0 || page > (s.kv - 1) / c.P) return false;
    w.ra = imax(p0, page * c.P);
    w.rb = imin(s.kv, (page + 1) * c.P);
    w.row0 = s.r0 - p0;
    w.off = w.ra - page * c.P;
    w.pid = c.table[(size_t)b * c.table_stride + page];
    w.placed = w.pid >= 0 && w.pid < c.n_pages;
    if (!w.placed && threadIdx.x == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
    return true;
}

// the scale of a page that holds `off` rows at scale `old` and gets rows of
// largest magnitude amax
__device__ __forceinline__ float joined_scale(float amax, float old, int off) {
    const float sc = pow2_scale(amax);
    return off > 0 ? (amax > 0.f ? fmaxf(sc, old) : old) : sc;
}
// sixteen stored values times f (old scale / new scale), rounded again
__device__ __forceinline__ void rescale16(uint8_t* at, float f) {
    uint4 w = *reinterpret_cast<uint4*>(at);
    uint32_t* wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a0, a1, a2, a3;
        f16x2_to_f32(e4m3x2_to_f16x2(wp[i] & 0xffffu), a0, a1);
        f16x2_to_f32(e4m3x2_to_f16x2(wp[i] >> 16), a2, a3);
        wp[i] = e4m3x2(a0 * f, a1 * f) | (e4m3x2(a2 * f, a3 * f) << 16);
    }
    *reinterpret_cast<uint4*>(at) = w;
}
// x / sc as e4m3.  A power of two (every scale this file makes; a pool filled
// elsewhere may hold others) divides exactly by a multiplication, and where no
// infinity is among the values (`inf`) the conversion needs no check (NaN stays NaN).
__device__ __forceinline__ void store_e4m3(uint8_t* dst, const LaneChunks& lc, const float (&x)[16], float sc, bool inf) {
    const uint32_t bits = __float_as_uint(sc);
    uint32_t w[4];
    const bool pow2 = (bits & 0x807fffffu) == 0u && bits >= 0x00800000u && bits <= 0x7e000000u;
    if (pow2 && !inf) {
        const float f = __uint_as_float(0x7f000000u - bits);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3x2_no_inf(x[4 * i] * f, x[4 * i + 1] * f) | (e4m3x2_no_inf(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16);
    } else if (pow2) {
        const float f = __uint_as_float(0x7f000000u - bits);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3x2(x[4 * i] * f, x[4 * i + 1] * f) | (e4m3x2(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3x2(x[4 * i] / sc, x[4 * i + 1] / sc) | (e4m3x2(x[4 * i + 2] / sc, x[4 * i + 3] / sc) << 16);
    }
    *reinterpret_cast<uint2*>(dst + lc.c0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(dst + lc.c1) = make_uint2(w[2], w[3]);
}

// Few rows a unit.  R rows of a head at a time, D / 16 lanes each, walk the page's
// new rows twice, first for the largest magnitude (e4m3 pages: the page's scale
// must cover them all before one is stored), then to store; a lane's first row stays in
// its registers between the two.  Bound by the chain of dependent loads: row
// range, length, page id, rows and old scale.  One row of 8 sequences takes 3.3 us, 6
// rows of 32 sequences 4.6 us (bf16 pages), most of it the launch and that chain.
template <int R>
__global__ void __launch_bounds__(256, 3) paged_append_step_kernel(const __grid_constant__ PagedAppendParams p) {
    pdl_wait();
    pdl_trigger();
    const PagedView& c = p.c;
    check_sequences(p);
    AppendUnit w;
    if (!find_unit(p, blockIdx.x, w)) return;

    const int tid = threadIdx.x, P = c.P;
    const int L = c.D / 16, t = tid % L, sub = tid / L % R, heads = 2 * c.Hkv + (p.q ? p.Hq : 0);
    const int hh = (int)blockIdx.y * ((int)blockDim.x / (L * R)) + tid / (L * R);
    const bool is_q = hh >= 2 * c.Hkv, is_v = !is_q && hh >= c.Hkv;
    const bool live = hh < heads && (is_q || w.placed), quant = live && !is_q && c.k_scale;
    const int h = is_q ? hh - 2 * c.Hkv : (is_v ? hh - c.Hkv : hh);
    const __nv_bfloat16* src = is_q ? p.q : (is_v ? p.v : p.k);
    const long long stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
    const bool rotate = p.cos_sin != nullptr && !is_v;
    const LaneChunks lc = lane_chunks(t, rotate ? p.rot : 0, p.interleaved);
    auto load = [&](int pos, float (&x)[16]) {
        const int row = w.row0 + pos;
        const int rp = p.pos ? p.pos[row] : pos;
        const bool in = rp >= 0 && rp < p.n_pos;
        if (rotate && !in && t == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
        load_rotated(src + (size_t)row * stride + (size_t)h * c.D, lc, rotate && in, p.cos_sin + (size_t)(in ? rp : 0) * p.rot,
                     p.rot, p.interleaved, x);
    };
    uint8_t* base = (is_v ? c.v : c.k) + (size_t)w.pid * c.page_bytes;
    float* sp = (is_v ? c.v_scale : c.k_scale) + (size_t)w.pid * c.Hkv + h;
    const int first = live ? w.ra + sub : w.rb;
    float x0[16], x[16], old = 0.f, amax = 0.f;
    if (quant && w.off > 0) old = *sp;
    if (first < w.rb) load(first, x0);
    if (live && !quant)
        for (int pos = first; pos < w.rb; pos += R) {
            if (pos > first) load(pos, x0);
            store_bf16(is_q ? p.q_out + ((size_t)(w.row0 + pos) * p.Hq + h) * c.D
                            : reinterpret_cast<__nv_bfloat16*>(base) + ((size_t)h * P + pos % P) * c.D,
                       lc, x0);
        }
    if (!c.k_scale) return;
    if (quant && first < w.rb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x0[i]));
        for (int pos = first + R; pos < w.rb; pos += R) {
            load(pos, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[i]));
        }
    }
    for (int o = 1; o < L * R; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncwarp();   // the old scale is read by every lane before one replaces it
    if (!quant) return;
    base += (size_t)h * P * c.D;
    const float sc = joined_scale(amax, old, w.off);
    if (w.off > 0 && sc > old)
        for (int r = sub; r < w.off; r += R) rescale16(base + (size_t)r * c.D + 16 * t, old / sc);
    for (int pos = first; pos < w.rb; pos += R) {
        if (pos > first) load(pos, x0);
        store_e4m3(base + (size_t)(pos % P) * c.D, lc, x0, sc, true);
    }
    if (t == 0 && sub == 0) *sp = sc;
}

// Many rows a unit.  A CTA of P D / (16 NP) threads holds a whole (page, head) in
// fp32 registers, NP rows a thread: one read, the largest magnitude over the
// CTA, one write.  It does `hg` heads one after the other, the next ones' rows on their
// way to shared memory, and keeps the cosines and sines of its rows for all of them.
// P D = 32768 leaves no registers for that (NP = 4).  Bound by HBM: a 32K prompt of
// 24 + 2 * 8 heads of 128 into e4m3 pages of 64 tokens takes 107 us, 5.8 TB/s (112 with
// every element checked for infinities twice, then 119 with kStages = 2 and 113 with 4,
// 186 with the angles read again for every head, 124 with the rows rotated again from
// shared memory instead of held and three CTAs an SM); walking the rows with the other
// kernel's loop took 268.
template <int NP>
__global__ void __launch_bounds__(512) paged_append_page_kernel(const __grid_constant__ PagedAppendParams p, int hg) {
    __shared__ uint32_t s_max[2][16];
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_wait();
    pdl_trigger();
    const PagedView& c = p.c;
    check_sequences(p);
    AppendUnit w;
    if (!find_unit(p, blockIdx.x, w)) return;

    constexpr bool kHold = NP <= 2;
    const int tid = threadIdx.x, P = c.P, D = c.D;
    const int L = D / 16, t = tid % L, G = (int)blockDim.x / L;
    const int heads = 2 * c.Hkv + (p.q ? p.Hq : 0);
    const int h0 = (int)blockIdx.y * hg, h1 = imin(h0 + hg, heads);
    const bool rope = p.cos_sin != nullptr, any_rot = rope && (h0 < c.Hkv || h1 > 2 * c.Hkv);
    // chunks of eight elements: the pairs of a lane lie in its two chunks, or (adjacent
    // pairs, rows that are not rotated) within each of them
    const LaneChunks plain{8 * t, D / 2 + 8 * t, -1};
    const LaneChunks turned = rope && !p.interleaved ? lane_chunks(t, p.rot, 0) : plain;
    const bool rot0 = rope && turned.c0 < p.rot, rot1 = rope && turned.c1 < p.rot;
    const int a0 = p.interleaved ? turned.c0 / 2 : turned.ang, a1 = p.interleaved ? turned.c1 / 2 : turned.ang + 4;

    int row[NP];
    bool has[NP], in[NP];
    const float* angles[NP];
    float cs[kHold ? NP : 1][16];
    auto load_angles = [&](const float* at, float (&o)[16]) {
        if (rot0) {
            *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(at + a0);
            *reinterpret_cast<float4*>(o + 8) = *reinterpret_cast<const float4*>(at + p.rot / 2 + a0);
        }
        if (rot1) {
            *reinterpret_cast<float4*>(o + 4) = *reinterpret_cast<const float4*>(at + a1);
            *reinterpret_cast<float4*>(o + 12) = *reinterpret_cast<const float4*>(at + p.rot / 2 + a1);
        }
    };
    // this thread's part of a head on its way: stage, row and chunk; no thread reads another's
    auto slot = [&](int stage, int j, int i) { return (unsigned)((((stage * NP + j) * 2 + i) * (int)blockDim.x + tid) * 16); };
    auto fetch = [&](int hh, int stage) {
        const bool q = hh >= 2 * c.Hkv, v = !q && hh >= c.Hkv;
        const __nv_bfloat16* src = q ? p.q + (size_t)(hh - 2 * c.Hkv) * D : (v ? p.v + (size_t)(hh - c.Hkv) * D : p.k + (size_t)hh * D);
        const long long stride = q ? p.q_stride : (v ? p.v_stride : p.k_stride);
        const LaneChunks& lc = v ? plain : turned;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const __nv_bfloat16* at = src + (size_t)row[j] * stride;
            cp_async16(smem_u32(smem) + slot(stage, j, 0), at + lc.c0, has[j] ? 16 : 0);
            cp_async16(smem_u32(smem) + slot(stage, j, 1), at + lc.c1, has[j] ? 16 : 0);
        }
    };
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int pos = w.ra + j * G + tid / L;
        has[j] = pos < w.rb;
        row[j] = w.row0 + (has[j] ? pos : w.ra);
    }
    for (int i = 0; i < kStages - 1; ++i) {
        if (h0 + i < h1) fetch(h0 + i, i);
        cp_async_commit();
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        in[j] = false;
        angles[j] = nullptr;
        if (any_rot && has[j]) {
            const int rp = p.pos ? p.pos[row[j]] : row[j] - w.row0;
            in[j] = rp >= 0 && rp < p.n_pos;
            if (!in[j] && t == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
            if (in[j]) {
                angles[j] = p.cos_sin + (size_t)rp * p.rot;
                if (kHold) load_angles(angles[j], cs[kHold ? j : 0]);
            }
        }
    }
    int par = 0, stage = 0;
    for (int hh = h0; hh < h1; ++hh) {
        const bool is_q = hh >= 2 * c.Hkv, is_v = !is_q && hh >= c.Hkv;
        const int h = is_q ? hh - 2 * c.Hkv : (is_v ? hh - c.Hkv : hh);
        const LaneChunks lc = is_v ? plain : turned;
        cp_async_wait<kStages - 2>();
        float x[NP][16];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(smem + slot(stage, j, 0)), x[j]);
            Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(smem + slot(stage, j, 1)), x[j] + 8);
        }
        if (hh + kStages - 1 < h1) fetch(hh + kStages - 1, stage > 0 ? stage - 1 : kStages - 1);
        cp_async_commit();
        stage = stage + 1 < kStages ? stage + 1 : 0;
        if (!is_v)
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (in[j]) {
                    float(&o)[16] = cs[kHold ? j : 0];
                    if (!kHold) load_angles(angles[j], o);
                    rotate16(x[j], o, p.interleaved, rot0, rot1);
                }
        if (is_q || !c.k_scale) {
            if (is_q || w.placed)
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    if (has[j]) {
                        __nv_bfloat16* dst =
                            is_q ? p.q_out + ((size_t)row[j] * p.Hq + h) * D
                                 : reinterpret_cast<__nv_bfloat16*>((is_v ? c.v : c.k) + (size_t)w.pid * c.page_bytes) +
                                       ((size_t)h * P + w.off + j * G + tid / L) * D;
                        store_bf16(dst, lc, x[j]);
                    }
            continue;
        }
        if (!w.placed) continue;
        float* sp = (is_v ? c.v_scale : c.k_scale) + (size_t)w.pid * c.Hkv + h;
        uint8_t* base = (is_v ? c.v : c.k) + (size_t)w.pid * c.page_bytes + (size_t)h * P * D;
        const float old = w.off > 0 ? *sp : 0.f;   // read by all before the barrier, written behind it
        float amax = 0.f;   // a maximum passes over NaN, and an infinity shows in it
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[j][i]));
        const bool inf = amax > 3.4028234663852886e38f;
        if (inf) {
            amax = 0.f;
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[j][i]));
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
        if (tid % 32 == 0) s_max[par][tid / 32] = top;
        __syncthreads();
        uint32_t all = 0;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) all = max(all, s_max[par][i]);
        par ^= 1;
        const float sc = joined_scale(__uint_as_float(all), old, w.off);
        if (w.off > 0 && sc > old)
            for (int r = tid / L; r < w.off; r += G) rescale16(base + (size_t)r * D + 16 * t, old / sc);
#pragma unroll
        for (int j = 0; j < NP; ++j)
            if (has[j]) store_e4m3(base + (size_t)(w.off + j * G + tid / L) * D, lc, x[j], sc, inf);
        if (tid == 0) *sp = sc;
    }
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
    const int heads = 2 * p.c.Hkv + p.Hq, per = rows / p.c.B;
    // n rows touch at most (n - 2) / P + 2 pages, one row one
    if (!row_start) p.per_seq = per > 1 ? (per - 2) / p.c.P + 2 : 1;
    const int units = row_start ? append_units(rows, p.c.B, p.c.P) : p.c.B * p.per_seq;
    cudaError_t e;
    // Many rows a page pay for a CTA that holds whole pages.  Its time hardly depends
    // on the rows, the other kernel's grows with them: 32 sequences, 64-token pages,
    // 40 heads of 128: 10.5 us at 4 rows and 11.0 at 12, against 4.5 and 7.7 (then 0.5 us
    // for every 4 rows).  When its CTAs fit at once, it wins earlier (8 sequences: 5.5 us
    // against 5.0 at 8 rows and 6.1 at 12; one: 3.1 against 3.3 at 1 row).
    const long long page_rows = (long long)p.c.B * p.c.P;
    if (rows * 3ll >= 2 * page_rows || (rows * 8ll >= page_rows && (long long)units * heads <= 768)) {
        const int lanes = p.c.P * p.c.D / 16, np = lanes > 1024 ? 4 : 2;
        // heads one CTA does in turn: up to 16, while two rounds of CTAs remain (a 32K prompt:
        // 4 heads 146 us, 8 heads 135, 16 heads 130, before rows went through shared memory)
        int hg = 1;
        while (hg < 16 && (long long)units * ((heads + 2 * hg - 1) / (2 * hg)) * (lanes / np) >= 152ll * 2048) hg *= 2;
        const size_t smem = (size_t)lanes * 32 * kStages;
        auto kern = np == 2 ? paged_append_page_kernel<2> : paged_append_page_kernel<4>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(32 * 2048 * kStages));
        if (e == cudaSuccess)
            e = masw_launch(kern, dim3(units, (heads + hg - 1) / hg), dim3(lanes / np), smem, (cudaStream_t)stream, 1, p, hg);
    } else {
        // Rows of a head side by side shorten the walk: 8 sequences of 4 rows 3.7 us against
        // 6.3.  They take four times the CTAs, too many at 256 sequences of fewer than 8 rows
        // (2 rows: 14.0 us against 9.5; 8 rows: 21 against 24).
        auto ctas_y = [&](int r) { return (heads * (p.c.D / 16) * r + 255) / 256; };
        const bool wide = per > 1 && (per >= 8 || (long long)units * ctas_y(4) <= 1024);
        e = masw_launch(wide ? paged_append_step_kernel<4> : paged_append_step_kernel<1>, dim3(units, ctas_y(wide ? 4 : 1)),
                        dim3(256), 0, (cudaStream_t)stream, 1, p);
    }
    if (e != cudaSuccess) return masw_set_error(nullptr, MASW_ECUDA, std::string("paged_append: ") + cudaGetErrorString(e));
    return MASW_OK;
}
