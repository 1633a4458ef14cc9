// What the paged-cache operators share: checked arguments, the parameters that
// describe a cache to a kernel, and the e4m3 conversions.
#pragma once

#include "masw_internal.cuh"

namespace masw {

// a paged cache as its kernels see it (strides in bytes)
struct PagedView {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;          // null: bf16 pages
    float* v_scale;
    const int* table;        // [batch][table_stride]
    long long page_bytes;    // between consecutive pages
    int n_pages, P, Hkv, D, B, table_stride;
    int cap;                 // tokens a table row can hold
};

// The rows of sequence b: [r0, r0 + n), at positions kv - n ..  `ok` is false
// (and n = 0) when the row range or the length cannot be what the caller meant.
struct SeqRows {
    int r0, n, kv;
    bool ok;
};
__host__ __device__ inline SeqRows seq_rows_of(int r0, int r1, int kv, int rows, int cap) {
    SeqRows s{r0, r1 - r0, kv, true};
    s.ok = r0 >= 0 && r1 >= r0 && r1 <= rows && kv >= 0 && kv <= cap;
    if (!s.ok) s.n = s.kv = 0;
    return s;
}
__device__ __forceinline__ SeqRows seq_rows(const int* row_start, const int* kv_len, int b, int rows, int B, int cap) {
    const int per = rows / B;
    const int r0 = row_start ? row_start[b] : b * per, r1 = row_start ? row_start[b + 1] : r0 + per;
    return seq_rows_of(r0, r1, kv_len[b], rows, cap);
}

// Units of an append: (sequence, touched page) pairs in a one-dimensional grid
// that the host can size without knowing the lengths.  n rows touch at most
// n / P + 2 pages, so sequence b owns units [r0 / P + 2 b, next): the next
// sequence's first unit lies at least n / P + 2 behind.
__host__ __device__ inline int append_unit_base(int r0, int b, int P) { return r0 / P + 2 * b; }
__host__ __device__ inline int append_units(int rows, int B, int P) { return rows / P + 2 * B; }

// smallest power of two s with amax <= 448 s, clamped to [2^-64, 2^119]; 1 for 0
__host__ __device__ inline int pow2_scale_exp(uint32_t amax_bits) {
    const int ex = (int)(amax_bits >> 23) - 127;
    const int e = (amax_bits & 0x7fffffu) <= 0x600000u ? ex - 8 : ex - 7;   // 448 = 1.75 * 2^8
    return amax_bits == 0u ? 0 : (e < -64 ? -64 : (e > 119 ? 119 : e));
}

// ---- how attention over few query rows is cut over CTAs --------------------
// The keys of one (sequence, kv head) pair come in tiles of 128.  All pairs'
// tiles form one line, sequence by sequence and head by head, and CTA c of C
// takes tiles [first_tile(c), first_tile(c + 1)) of it: every CTA gets the same
// number of tiles (give or take one; CTAs behind the last tile get none) whatever
// the lengths are.  A pair that is cut leaves one partial result for each CTA that holds a piece of it: in that
// CTA's slot 0 if the piece is the CTA's first, else in its slot 1 (its last).
// Where a CTA has few tiles anyway, a second piece (its Q, the first maxima, the end's
// sums and outputs: ~3.5 us) costs more than uneven shares: then every pair gets
// pair_ctas CTAs of its own, and CTA pair * pair_ctas + i takes tiles
// [part_first(i), part_first(i + 1)) of the pair, possibly none, and uses slot 0.
constexpr int kTile = 128;
constexpr int kUneven = 3;   // tiles that a CTA may have beyond the even share
struct TileRange {
    int lo, hi;   // visible keys of the sequence's rows: [lo, hi)
    int t0, nt;   // first tile and number of tiles (at least one: it writes the outputs)
};
__host__ __device__ inline TileRange tile_range(int n, int kv, int window) {
    TileRange r{0, kv, 0, 0};
    if (n < 1) return r;
    if (window > 0 && kv - n - window + 1 > 0) r.lo = kv - n - window + 1;
    r.t0 = r.lo / kTile;
    r.nt = (r.hi + kTile - 1) / kTile - r.t0;
    if (r.nt < 1) r.nt = 1;
    return r;
}
// tiles of every CTA: total / C, one more for the first total % C
__host__ __device__ inline int first_tile(int c, int total, int C) {
    const int q = total / C, rem = total - q * C;
    return c * q + (c < rem ? c : rem);
}
__host__ __device__ inline int tile_owner(int t, int total, int C) {
    const int q = total / C, rem = total - q * C;
    return t < rem * (q + 1) ? t / (q + 1) : rem + (t - rem * (q + 1)) / q;
}

// CTAs of every pair, or 0: the line is cut evenly.  longest: tiles of the longest pair
__host__ __device__ inline int pair_ctas(int pairs, int longest, int total, int C) {
    const int s = pairs <= C ? C / pairs : 0;
    return s > 0 && (longest + s - 1) / s <= total / C + kUneven ? s : 0;
}
__host__ __device__ inline int part_first(int i, int nt, int s) {
    return nt > s ? (int)((long long)i * nt / s) : (i < nt ? i : nt);   // the first min(nt, s) parts have tiles
}

#ifdef __CUDACC__
__device__ __forceinline__ float pow2_scale(float amax) {
    return __uint_as_float((uint32_t)(pow2_scale_exp(__float_as_uint(amax)) + 127) << 23);
}
// |x|, or 0 for infinities and NaN
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4028234663852886e38f ? a : 0.f;
}
// two fp32 values -> e4m3 (round to nearest even, lo in bits 0..7); what is not
// finite becomes NaN (the conversion itself would saturate an infinity)
__device__ __forceinline__ uint32_t e4m3x2_no_inf(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    lo = fabsf(lo) <= 3.4028234663852886e38f ? lo : __int_as_float(0x7fffffff);
    hi = fabsf(hi) <= 3.4028234663852886e38f ? hi : __int_as_float(0x7fffffff);
    return e4m3x2_no_inf(lo, hi);
}
// two e4m3 values (bits 0..7 and 8..15) -> f16x2
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float& lo, float& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
}
#endif

}  // namespace masw

// Argument checks shared by the paged calls; fills `view`.  0 or a status with
// the message set.
int masw_paged_view(const masw_paged_t* cache, const char* who, masw::PagedView* view);
