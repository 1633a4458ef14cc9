// Attention of few query rows over a paged cache (decode and verify): up to 32
// rows (query token x query head of the group) of a (sequence, kv head) pair.
//
// What bounds it is reading the cache once: 2 D bytes a key and head in e4m3,
// 4 D in bf16, for 4 D flops a row.  So every SM runs one CTA that streams tiles
// of 128 keys by TMA through a ring of shared-memory stages, and everything else
// hides behind that stream:
//   * one line of tiles over all pairs, cut into equal shares (TileRange), so
//     ragged batches load every SM alike; a merge kernel joins the cut pairs;
//   * S^T = K Q^T on the tensor cores with the 128 keys as M and the rows as N:
//     a thread owns one key and finds its score of every row in its TMEM lane.
//     No reduction over keys happens in the loop: sums stay per thread until a
//     pair ends, and the running maximum is only checked ("is any score more than
//     2^8 above the reference?", one barrier with a vote) and moved, with O
//     rescaled, when it is -- usually in a pair's first tiles only;
//   * O^T += V^T P^T with head_dim as M: V is read as it lies in the page;
//   * e4m3 pages enter the tensor cores as they are.  Q is split into two e4m3
//     terms (q1 + q2 / 16, exact for bf16 unless an element is 2^-21 of the
//     largest) and the weights into three (p1 + p2 / 16 + p3 / 256 of their fp16
//     value, 2^-12 relative): the terms lie side by side in N, so a tile of K or
//     V is read by the tensor core once for all of them.  The scale of a key's
//     page multiplies its scores; the scale of its value's page enters the
//     exponent, 2^(s + log2 scale - reference), and the sum takes it out again;
//   * bf16 pages: weights as two bf16 terms (2^-17).
// Rows behind the end of a sequence never count: their scores are masked, and
// their V rows are zeroed in shared memory (0 x NaN is NaN in a matrix product).
//
// Warps 0-3: softmax and outputs; 4: issues S; 5: issues O; 6: page ids, scales
// and TMA; 7: loads and splits Q for the next pair.  Hand-offs are mbarriers;
// every wait is bounded.
#include "masw_paged_attn.cuh"

namespace masw {
namespace rows {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kMeta = 16;    // tiles of scales kept: more than a stage ring's tiles in flight

template <bool E4, int D, int NP>
struct Cfg {
    static constexpr int kES = E4 ? 1 : 2;
    static constexpr int kRB = D * kES;                         // bytes of a key's row
    static constexpr int kPanels = kRB > 128 ? 2 : 1;           // 128-byte column panels of a tile
    static constexpr int kPB = kRB / kPanels;                   // bytes of a row in a panel
    static constexpr uint32_t kPanel = kTile * kPB;
    static constexpr uint32_t kTileB = kTile * kRB;
    static constexpr uint32_t kSwz = kPB == 128 ? 2 : 4;        // 128- or 64-byte swizzle
    static constexpr uint32_t kAtom = 8 * kPB;                  // 8 rows
    static constexpr int kSN = E4 ? 2 * NP : (NP < 16 ? 16 : NP);            // columns of S^T
    static constexpr int kPN = E4 ? (NP == 8 ? 32 : 3 * NP) : 2 * NP;        // columns of P^T and O^T
    static constexpr int kTerms = E4 ? 3 : 2;
    static constexpr uint32_t kPBuf = kTile * kPN * kES;
    static constexpr uint32_t kQBuf = kSN * kRB;
    static constexpr bool kWide = !E4 && D == 128;              // 32 KB tiles: three stages
    static constexpr int kST = kWide ? 3 : (kRB == 128 ? 5 : 8);
    static constexpr int kPBufs = kWide && NP == 32 ? 1 : 2;
    static constexpr int kQBufs = kWide && NP == 32 ? 1 : 2;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kST * kTileB;
    static constexpr uint32_t kOffP = kOffV + kST * kTileB;
    static constexpr uint32_t kOffQ = kOffP + kPBufs * kPBuf;
    static constexpr uint32_t kOffSeq = kOffQ + kQBufs * kQBuf;               // pre[B + 1], kv, n, r0
    static constexpr uint32_t kOffMeta = kOffSeq + 4 * (4 * MASW_MAX_BATCH + 4);
    static constexpr uint32_t kOffRed = kOffMeta + (E4 ? kMeta * 8 * 16 : 0);  // [2][4][NP] floats
    static constexpr uint32_t kOffQs = kOffRed + 2 * 4 * NP * 4;                   // scale of Q per buffer
    static constexpr uint32_t kOffBar = kOffQs + 16;
    // barriers
    static constexpr int kKFull = 0, kKFree = kST, kVFull = 2 * kST, kVFree = 3 * kST, kMetaBar = 4 * kST;
    static constexpr int kSFull = kMetaBar + (E4 ? kMeta : 0), kSFree = kSFull + 2, kPFull = kSFree + 2, kPFree = kPFull + 2;
    static constexpr int kQFull = kPFree + 2, kQFree = kQFull + 2, kDone = kQFree + 2, kBars = kDone + 2;
    static constexpr uint32_t kSmem = kOffBar + 8 * kBars + 16;               // + TMEM address, abort flag
    static constexpr uint32_t kColO = 2 * kSN;
    static constexpr uint32_t kCols = 2 * kSN + kPN <= 64 ? 64 : (2 * kSN + kPN <= 128 ? 128 : 256);
    static constexpr uint32_t kType = E4 ? 0 : 1;               // operand type field: e4m3 / bf16
    static constexpr uint32_t kBase = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(kTile >> 4) << 24);
    static constexpr uint32_t kIdescS = kBase | ((uint32_t)(kSN >> 3) << 17);
    static constexpr uint32_t kIdescO = kBase | (1u << 15) | (1u << 16) | ((uint32_t)(kPN >> 3) << 17);
    // the exponent's reference lies this far below the largest score, and may be
    // exceeded by 2^8: e4m3 weights reach 256 (of 448)
    static constexpr float kHead = E4 ? 5.f : 0.f;
    static_assert(kSmem + 1024 <= 232448, "shared memory");
    static_assert(kST + 2 < kMeta, "scales would be overwritten");
};

// A CTA's walk over its tiles, piece by piece (a piece: tiles of one pair).
struct Walk {
    int t, t1;               // tiles of the line left: [t, t1)
    int b, h, tile, nt;      // the piece: sequence, kv head, first tile, number of tiles
    bool whole, first;       // the piece is its whole pair; the CTA's first
};

__device__ __forceinline__ bool next_piece(Walk& w, const int* pre, int B, int Hkv, const int* kv, const int* n, int window) {
    if (w.t >= w.t1) return false;
    while (w.b + 1 < B && pre[w.b + 1] <= w.t) ++w.b;
    const int per = (pre[w.b + 1] - pre[w.b]) / Hkv, in = w.t - pre[w.b];
    w.h = in / per;
    const int at = in - w.h * per;
    w.tile = tile_range(n[w.b], kv[w.b], window).t0 + at;
    w.nt = imin(per - at, w.t1 - w.t);
    w.whole = at == 0 && w.nt == per;
    w.t += w.nt;
    return true;
}

__device__ __forceinline__ bool bar_or(bool x) {   // vote over the 128 softmax threads
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_softmax() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
// 16 (h - e) for a pair: what e4m3 left of it, exactly
__device__ __forceinline__ uint32_t rest16(uint32_t h, uint32_t e) {
    uint32_t a, r;
    const uint32_t s = 0x4C004C00u, ms = 0xCC00CC00u;   // 16, -16
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(h), "r"(s));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(e), "r"(ms), "r"(a));
    return r;
}

template <bool E4, int D, int NP>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ PagedAttnParams p) {
    using C = Cfg<E4, D, NP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sb = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* err_sink = reinterpret_cast<int*>(tslot + 2);
    int* pre = reinterpret_cast<int*>(smem + C::kOffSeq);
    int* s_kv = pre + MASW_MAX_BATCH + 1;
    int* s_n = s_kv + MASW_MAX_BATCH;
    int* s_r0 = s_n + MASW_MAX_BATCH;
    float4* meta = reinterpret_cast<float4*>(smem + C::kOffMeta);   // [kMeta][8]: K scale, log2 V scale, 1 / V scale
    float* red = reinterpret_cast<float*>(smem + C::kOffRed);       // [4][NP] row maxima of the warps
    float* sums = red + 4 * NP;                                     // [4][NP] row sums of the warps
    float* qscale = reinterpret_cast<float*>(smem + C::kOffQs);
    auto bar_at = [&](int i) { return sb + C::kOffBar + 8u * (uint32_t)i; };
    const PagedView& c = p.c;
    const int B = c.B, Hkv = c.Hkv, G = p.G;

    if (sb & 1023u) {   // the swizzled layouts need it
        if (tid == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < C::kBars; ++i)
            mbar_init(bars + i, i >= C::kQFree && i < C::kQFree + 2                                                         ? 5
                                : (i >= C::kSFree && i < C::kSFree + 2) || (i >= C::kPFull && i < C::kPFull + 2) ? 4
                                                                                                                 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    int* const err = p.status ? p.status : err_sink;
    const int total = make_line<kThreads>(p, pre, s_kv, s_n, s_r0, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    Walk walk;
    walk.t = first_tile(blockIdx.x, total, gridDim.x);
    walk.t1 = first_tile(blockIdx.x + 1, total, gridDim.x);
    {   // the sequence of the first tile
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= walk.t) lo = mid;
            else hi = mid;
        }
        walk.b = lo;
    }
    auto wait = [&](int bar, int phase) { return wait_or_abort(bars + bar, (uint32_t)phase & 1u, abort_flag, err); };
    bool ok = true;

    if (warp == 4) {
        // ---------------- S^T = K Q^T ----------------
        if (lane == 0) {
            int i = 0, piece = 0;
            while (ok && next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
                const int qb = piece % C::kQBufs;
                ok = wait(C::kQFull + qb, piece / C::kQBufs);
                const uint64_t bq = smem_desc(sb + C::kOffQ + qb * C::kQBuf, 128, (C::kRB / 16) * 128, 0);
                for (int j = 0; ok && j < walk.nt; ++j, ++i) {
                    const int st = i % C::kST, sbuf = i & 1;
                    ok = wait(C::kKFull + st, i / C::kST) && (i < 2 || wait(C::kSFree + sbuf, i / 2 - 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ak = smem_desc(sb + C::kOffK + st * C::kTileB, 16, C::kAtom, C::kSwz);
#pragma unroll
                    for (int kk = 0; kk < C::kRB / 32; ++kk) {
                        const uint64_t a = ak + (uint64_t)(((kk / (C::kPB / 32)) * C::kPanel + (kk % (C::kPB / 32)) * 32) >> 4);
                        const uint64_t b = bq + (uint64_t)((kk * 256) >> 4);
                        if (E4) umma_f8(tmem + sbuf * C::kSN, a, b, C::kIdescS, kk > 0);
                        else umma_bf16(tmem + sbuf * C::kSN, a, b, C::kIdescS, kk > 0);
                    }
                    umma_commit(bar_at(C::kSFull + sbuf));
                    umma_commit(bar_at(C::kKFree + st));
                    if (j + 1 == walk.nt) umma_commit(bar_at(C::kQFree + qb));
                }
                ++piece;
            }
            // nothing may arrive on a barrier after the CTA ended
            if (ok && i > 0) ok = wait(C::kKFree + (i - 1) % C::kST, (i - 1) / C::kST) && wait(C::kQFree + (piece - 1) % C::kQBufs, (piece - 1) / C::kQBufs);
            if (!ok) {   // let the matrix products in flight end before the CTA does
                *abort_flag = 1;
                umma_commit(bar_at(C::kDone));
                mbar_wait(bars + C::kDone, 0, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ---------------- O^T += V^T P^T ----------------
        if (lane == 0) {
            int i = 0;
            while (ok && next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
                for (int j = 0; ok && j < walk.nt; ++j, ++i) {
                    const int st = i % C::kST, pb = i % C::kPBufs;
                    ok = wait(C::kPFull + pb, i / C::kPBufs) && wait(C::kVFull + st, i / C::kST);
                    if (!ok) break;
                    tc_fence_after();
                    // head_dim 64: the second half of the 128 M rows repeats the first
                    // (a leading offset of 0); head_dim 128 in bf16: the second panel
                    const uint64_t av = smem_desc(sb + C::kOffV + st * C::kTileB, C::kPanels == 2 ? C::kPanel : 0, C::kAtom, C::kSwz);
                    const uint64_t bp = smem_desc(sb + C::kOffP + pb * C::kPBuf, 128, 2048, 0);
                    constexpr int kKeys = 32 / C::kES;   // keys of one matrix instruction
#pragma unroll
                    for (int kk = 0; kk < kTile / kKeys; ++kk) {
                        const uint64_t a = av + (uint64_t)((kk * kKeys * C::kPB) >> 4);
                        const uint64_t b = bp + (uint64_t)((kk * kKeys * 16) >> 4);
                        if (E4) umma_f8(tmem + C::kColO, a, b, C::kIdescO, j > 0 || kk > 0);
                        else umma_bf16(tmem + C::kColO, a, b, C::kIdescO, j > 0 || kk > 0);
                    }
                    umma_commit(bar_at(C::kPFree + pb));
                    umma_commit(bar_at(C::kVFree + st));
                }
            }
            if (ok && i > 0) ok = wait(C::kVFree + (i - 1) % C::kST, (i - 1) / C::kST);
            if (!ok) {
                *abort_flag = 1;
                umma_commit(bar_at(C::kDone + 1));
                mbar_wait(bars + C::kDone + 1, 0, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ---------------- page ids, scales, TMA ----------------
        // A lane holds the page of one box (at most 128 rows of a page); a batch
        // is up to 32 boxes of a piece.  The next batch's page ids are loaded
        // while the current one is issued, and its scales once they are there.
        const int box = imin(c.P, kTile), bpt = kTile / box, bt = 32 / bpt;   // boxes a tile, tiles a batch
        Walk w = walk;
        int left = 0, at = 0;            // tiles of the piece not yet in a batch, and the first of them
        struct Batch { int h, tile, nt, pid; bool in; float ks, vs; };
        auto next_batch = [&](Batch& x) {
            x.nt = 0;
            x.in = false;
            if (left == 0) {
                if (!next_piece(w, pre, B, Hkv, s_kv, s_n, p.window)) return;
                left = w.nt;
                at = w.tile;
            }
            x.h = w.h;
            x.tile = at;
            x.nt = imin(left, bt);
            at += x.nt;
            left -= x.nt;
            const TileRange r = tile_range(s_n[w.b], s_kv[w.b], p.window);
            const int key = x.tile * kTile + lane * box;
            x.in = lane < x.nt * bpt && key < r.hi && (key / c.P + 1) * c.P > r.lo;
            x.pid = x.in ? __ldg(c.table + (size_t)w.b * c.table_stride + key / c.P) : 0;
        };
        auto check_and_scale = [&](Batch& x) {
            if (x.in && (x.pid < 0 || x.pid >= c.n_pages)) {
                atomicExch(err, MASW_EINVAL);
                x.pid = 0;
            }
            x.ks = x.vs = 1.f;
            if (E4 && x.in) {
                x.ks = __ldg(c.k_scale + (size_t)x.pid * Hkv + x.h);
                x.vs = __ldg(c.v_scale + (size_t)x.pid * Hkv + x.h);
            }
        };
        Batch cur, nxt;
        int i = 0;
        next_batch(cur);
        next_batch(nxt);
        check_and_scale(cur);
        while (ok && cur.nt > 0) {
            check_and_scale(nxt);
            Batch nn;
            next_batch(nn);
            for (int j = 0; ok && j < cur.nt; ++j, ++i) {
                const int st = i % C::kST;
                const bool mine = lane / bpt == j && cur.in;
                const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
                const uint32_t bytes = (uint32_t)boxes * box * C::kRB;
                const int row = ((cur.tile + j) * kTile + (lane % bpt) * box) & (c.P - 1);
                const uint32_t dst = (uint32_t)st * C::kTileB + (uint32_t)((lane % bpt) * box * C::kPB);
                if (i >= C::kST) ok = __all_sync(0xffffffffu, wait(C::kKFree + st, i / C::kST - 1));
                if (!ok) break;
                if (E4 && lane / bpt == j)
                    meta[(i % kMeta) * 8 + lane % bpt] =
                        make_float4(cur.ks, cur.vs == 1.f ? 0.f : __log2f(cur.vs), __frcp_rn(cur.vs), 0.f);
                __syncwarp();
                if (lane == 0) {
                    if (E4) mbar_arrive(bar_at(C::kMetaBar + i % kMeta));
                    mbar_expect_tx(bars + C::kKFull + st, bytes);
                }
                __syncwarp();
                if (mine)
#pragma unroll
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        tma_load_4d(sb + C::kOffK + dst + pn * C::kPanel, &p.tm_k, pn * C::kPB / C::kES, row, cur.h, cur.pid,
                                    bar_at(C::kKFull + st));
                if (i >= C::kST) ok = __all_sync(0xffffffffu, wait(C::kVFree + st, i / C::kST - 1));
                if (!ok) {   // the K tile was issued, its V tile was not
                    mbar_wait(bars + C::kKFull + st, (uint32_t)(i / C::kST) & 1u, nullptr);
                    break;
                }
                if (lane == 0) mbar_expect_tx(bars + C::kVFull + st, bytes);
                __syncwarp();
                if (mine)
#pragma unroll
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        tma_load_4d(sb + C::kOffV + dst + pn * C::kPanel, &p.tm_v, pn * C::kPB / C::kES, row, cur.h, cur.pid,
                                    bar_at(C::kVFull + st));
            }
            cur = nxt;
            nxt = nn;
        }
        // after a wait gave up, and at the end: no copy may be in flight when the CTA ends
        if (!ok) *abort_flag = 1;
        for (int k = imax(0, i - C::kST); k < i; ++k) {
            mbar_wait(bars + C::kKFull + k % C::kST, (uint32_t)(k / C::kST) & 1u, nullptr);
            mbar_wait(bars + C::kVFull + k % C::kST, (uint32_t)(k / C::kST) & 1u, nullptr);
        }
        __syncwarp();
    } else if (warp == 7) {
        // ---------------- Q of the next pair ----------------
        constexpr int kLanes = D / 8, kPer = 32 / kLanes, kPass = NP / kPer;   // lanes a row, rows a pass
        int piece = 0;
        while (ok && next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
            const int nq = s_n[walk.b] * G, r0 = s_r0[walk.b];
            uint4 x[kPass];
            float amax = 0.f;
#pragma unroll
            for (int s = 0; s < kPass; ++s) {
                const int r = s * kPer + lane / kLanes;
                x[s] = make_uint4(0u, 0u, 0u, 0u);
                if (r < nq)
                    x[s] = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)(r0 + r / G) * p.q_stride +
                                                                (size_t)(walk.h * G + r % G) * D) +
                                 lane % kLanes);
            }
            const int qb = piece % C::kQBufs;
            float inv = 1.f;
            if (E4) {
#pragma unroll
                for (int s = 0; s < kPass; ++s) {
                    float f[8];
                    Elem<__nv_bfloat16>::unpack(x[s], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(f[e]));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                inv = 1.f / pow2_scale(amax);
            }
            if (piece >= C::kQBufs) ok = __all_sync(0xffffffffu, wait(C::kQFree + qb, piece / C::kQBufs - 1));
            if (!ok) break;
            const uint32_t qbase = sb + C::kOffQ + qb * C::kQBuf;
            // K-major core matrices of 8 rows x 16 bytes, consecutive along the row
            auto at = [&](int row, int byte) {
                return qbase + (uint32_t)((row >> 3) * (C::kRB / 16) * 128 + (byte >> 4) * 128 + (row & 7) * 16 + (byte & 15));
            };
#pragma unroll
            for (int s = 0; s < kPass; ++s) {
                const int r = s * kPer + lane / kLanes, e0 = (lane % kLanes) * 8;
                if (E4) {
                    float f[8];
                    Elem<__nv_bfloat16>::unpack(x[s], f);
                    uint32_t w1[4], w2[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float a = f[e] * inv, b = f[e + 1] * inv;
                        const uint32_t q1 = e4m3x2(a, b);
                        float a1, b1;
                        f16x2_to_f32(e4m3x2_to_f16x2(q1), a1, b1);
                        w1[e / 2] = q1;
                        w2[e / 2] = e4m3x2((a - a1) * 16.f, (b - b1) * 16.f);
                    }
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at(r, e0)), "r"(w1[0] | (w1[1] << 16)), "r"(w1[2] | (w1[3] << 16)) : "memory");
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at(NP + r, e0)), "r"(w2[0] | (w2[1] << 16)), "r"(w2[2] | (w2[3] << 16)) : "memory");
                } else {
                    st_shared_v4(at(r, e0 * 2), x[s].x, x[s].y, x[s].z, x[s].w);
                    if (NP < 16) st_shared_v4(at(NP + r, e0 * 2), 0u, 0u, 0u, 0u);
                }
            }
            if (lane == 0) qscale[qb] = p.scale_log2 / inv;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_at(C::kQFull + qb));
            ++piece;
        }
        if (!ok) *abort_flag = 1;
    } else {
        // ---------------- softmax: thread tid owns key tid of each tile ----------------
        // After a wait gave up these warps go on to the end of their tiles (every
        // later wait returns at once), so that they meet at their barriers.
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const uint32_t t_o = tmem + C::kColO + lane_off;
        int i = 0, piece = 0;
        bool first = true;
        while (next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
            const int b = walk.b, n = s_n[b], kv = s_kv[b], nq = n * G, q_pos = kv - n;
            const TileRange range = tile_range(n, kv, p.window);
            const int qb = piece % C::kQBufs;
            // keys that every row sees: [all_lo, all_hi)
            const int all_hi = q_pos + 1, all_lo = p.window > 0 ? imax(0, kv - p.window) : 0;
            float mref[NP], l[NP];
#pragma unroll
            for (int r = 0; r < NP; ++r) {
                mref[r] = -1e30f;
                l[r] = 0.f;
            }
            ok &= __all_sync(0xffffffffu, wait(C::kQFull + qb, piece / C::kQBufs)) != 0;
            const float qs = qscale[qb];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_at(C::kQFree + qb));
            for (int j = 0; j < walk.nt; ++j, ++i) {
                const int sbuf = i & 1;
                ok &= __all_sync(0xffffffffu, wait(C::kSFull + sbuf, i / 2)) != 0;
                tc_fence_after();
                float x[NP];
                {
                    uint32_t sv[C::kSN];
                    const uint32_t ts = tmem + sbuf * C::kSN + lane_off;
                    if constexpr (C::kSN == 16) {
                        tmem_ld16(ts, sv);
                    } else {
#pragma unroll
                        for (int q = 0; q < C::kSN / 32; ++q)
                            tmem_ld32(ts + q * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + q * 32));
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < NP; ++r)
                        x[r] = E4 ? fmaf(__uint_as_float(sv[NP + r]), 0.0625f, __uint_as_float(sv[r])) : __uint_as_float(sv[r]);
                }
                float ks = qs, lvs = 0.f, ivs = 1.f;
                const int tile0 = (walk.tile + j) * kTile, key = tile0 + tid;
                if (E4) {
                    ok &= __all_sync(0xffffffffu, wait(C::kMetaBar + i % kMeta, i / kMeta)) != 0;
                    const float4 mt = meta[(i % kMeta) * 8 + (c.P >= kTile ? 0 : tid / c.P)];
                    ks *= mt.x;
                    lvs = mt.y;
                    ivs = mt.z;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kSFree + sbuf));
                const bool masked = tile0 < all_lo || tile0 + kTile > all_hi;
                const bool seen = key >= range.lo && key < range.hi;   // by some row
                uint32_t see = 0xffffffffu;                            // by which rows
                if (masked) {
                    if (!seen) {
                        ks = 1.f;
                        lvs = 0.f;
                        ivs = 1.f;
                    }
                    see = 0u;
                    int pos = q_pos, g = 0;
                    for (int r = 0; r < nq; ++r) {
                        if (seen && key <= pos && (p.window <= 0 || key > pos - p.window)) see |= 1u << r;
                        if (++g == G) {
                            g = 0;
                            ++pos;
                        }
                    }
                    // a V row that no row sees must not reach the product
                    const int st = i % C::kST;
                    ok &= __all_sync(0xffffffffu, wait(C::kVFull + st, i / C::kST)) != 0;
                    if (!seen) {
#pragma unroll
                        for (int pn = 0; pn < C::kPanels; ++pn)
#pragma unroll
                            for (int q = 0; q < C::kPB / 16; ++q)
                                st_shared_v4(sb + C::kOffV + st * C::kTileB + pn * C::kPanel + tid * C::kPB + q * 16, 0u, 0u, 0u, 0u);
                    }
                }
                // weights relative to the reference of each row; the reference moves
                // when a score exceeds it by more than 2^8
                float mx = -INFINITY;
                float a[NP];
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    a[r] = fmaf(x[r], ks, lvs - mref[r]);
                    if (masked) a[r] = (see >> r) & 1u ? a[r] : -INFINITY;
                    mx = fmaxf(mx, a[r]);
                }
                if (bar_or(mx > 8.f)) {
#pragma unroll
                    for (int r = 0; r < NP; ++r) {
                        float s = (see >> r) & 1u ? fmaf(x[r], ks, lvs) : -INFINITY;
#pragma unroll
                        for (int o = 16; o; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
                        if (lane == 0) red[warp * NP + r] = s;
                    }
                    bar_softmax();
                    if (j > 0) {
                        // O holds tiles 0..j-1 of the piece once the last product is done
                        const int pb = (i - 1) % C::kPBufs;
                        ok &= __all_sync(0xffffffffu, wait(C::kPFree + pb, (i - 1) / C::kPBufs)) != 0;
                        tc_fence_after();
                    }
                    float alpha[NP];
#pragma unroll
                    for (int r = 0; r < NP; ++r) {
                        const float top = fmaxf(fmaxf(red[r], red[NP + r]), fmaxf(red[2 * NP + r], red[3 * NP + r])) - C::kHead;
                        const float nm = fmaxf(mref[r], top);
                        alpha[r] = ex2_approx(mref[r] - nm);
                        l[r] *= alpha[r];
                        mref[r] = nm;
                        a[r] = (see >> r) & 1u ? fmaf(x[r], ks, lvs - nm) : -INFINITY;
                    }
                    if (j > 0) {
#pragma unroll
                        for (int q = 0; q < C::kPN / 16; ++q) {
                            uint32_t ov[16];
                            tmem_ld16(t_o + q * 16, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha[(q * 16 + e) % NP]);
                            tmem_st16(t_o + q * 16, ov);
                        }
                        tmem_wait_st();
                    }
                }
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    a[r] = ex2_approx(a[r]);
                    l[r] = fmaf(a[r], ivs, l[r]);
                }
                const int pb = i % C::kPBufs;
                if (i >= C::kPBufs) {
                    ok &= __all_sync(0xffffffffu, wait(C::kPFree + pb, i / C::kPBufs - 1)) != 0;
                    tc_fence_after();
                }
                // this key's weights of all rows: the terms side by side, in 16-byte
                // chunks of core matrices (8 keys x 16 bytes)
                const uint32_t pw = sb + C::kOffP + pb * C::kPBuf + (uint32_t)((tid >> 3) * 128 + (tid & 7) * 16);
                if constexpr (E4) {
                    uint32_t w[3][NP / 4];
#pragma unroll
                    for (int r = 0; r < NP; r += 4) {
                        uint32_t h0 = cvt_f16x2(a[r], a[r + 1]), h1 = cvt_f16x2(a[r + 2], a[r + 3]);
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const uint32_t e0 = cvt_e4m3x2_f16x2(h0), e1 = cvt_e4m3x2_f16x2(h1);
                            w[k][r / 4] = e0 | (e1 << 16);
                            if (k < 2) {
                                h0 = rest16(h0, e4m3x2_to_f16x2(e0));
                                h1 = rest16(h1, e4m3x2_to_f16x2(e1));
                            }
                        }
                    }
                    if constexpr (NP == 8) {
                        st_shared_v4(pw, w[0][0], w[0][1], w[1][0], w[1][1]);
                        st_shared_v4(pw + 2048, w[2][0], w[2][1], 0u, 0u);
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k)
#pragma unroll
                            for (int q = 0; q < NP / 16; ++q)
                                st_shared_v4(pw + (k * (NP / 16) + q) * 2048, w[k][4 * q], w[k][4 * q + 1], w[k][4 * q + 2], w[k][4 * q + 3]);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < NP; r += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = a[r + 2 * e], v = a[r + 2 * e + 1];
                            hi[e] = pack_bf16(u, v);
                            lo[e] = pack_bf16(u - bf16lo(hi[e]), v - bf16hi(hi[e]));
                        }
                        st_shared_v4(pw + (r / 8) * 2048, hi[0], hi[1], hi[2], hi[3]);
                        st_shared_v4(pw + (NP / 8 + r / 8) * 2048, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kPFull + pb));
            }
            // the pair's (or piece's) sums over all keys, then O
#pragma unroll
            for (int r = 0; r < NP; ++r) {
#pragma unroll
                for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
                if (lane == 0) sums[warp * NP + r] = l[r];
            }
            bar_softmax();
#pragma unroll
            for (int r = 0; r < NP; ++r) l[r] = sums[r] + sums[NP + r] + sums[2 * NP + r] + sums[3 * NP + r];
            ok &= __all_sync(0xffffffffu, wait(C::kPFree + (i - 1) % C::kPBufs, (i - 1) / C::kPBufs)) != 0;
            tc_fence_after();
            float o[NP];
            {
                uint32_t ov[C::kPN];
#pragma unroll
                for (int q = 0; q < C::kPN / 16; ++q) tmem_ld16(t_o + q * 16, *reinterpret_cast<uint32_t(*)[16]>(ov + q * 16));
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    o[r] = __uint_as_float(ov[r]);
                    if (E4)
                        o[r] += fmaf(__uint_as_float(ov[2 * NP + r]), 0.00390625f, 0.0625f * __uint_as_float(ov[NP + r]));
                    else
                        o[r] += __uint_as_float(ov[NP + r]);
                }
            }
            tc_fence_before();
            if (walk.whole) {
                int tok = s_r0[b], g = 0;
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    if (r < nq) {
                        const size_t row = (size_t)tok * p.Hq + walk.h * G + g;
                        if (tid < D) store_out(p, row * D + tid, l[r] == 0.f ? 0.f : o[r] / l[r]);
                        if (tid == 0 && p.lse)
                            p.lse[row] = l[r] == 0.f ? -INFINITY : (mref[r] + __log2f(l[r])) * 0.6931471805599453f;
                        if (++g == G) {
                            g = 0;
                            ++tok;
                        }
                    }
                }
            } else {
                float* part = p.part + ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * kRowsMax * (D + 2);
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    if (r < nq) {
                        if (tid < D) __stcg(part + r * D + tid, o[r]);
                        if (tid == 0) {
                            __stcg(part + kRowsMax * D + r, l[r] == 0.f ? -INFINITY : mref[r]);
                            __stcg(part + kRowsMax * (D + 1) + r, l[r]);
                        }
                    }
                }
            }
            first = false;
            ++piece;
            bar_softmax();   // the sums were read
        }
        if (!ok) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
    }
}

// Joins the pieces of the pairs that were cut.  CTA (pair, 4 rows); thread d
// owns output element d.
template <int D>
__global__ void __launch_bounds__(128) rows_merge_kernel(const __grid_constant__ PagedAttnParams p, int n_cta) {
    __shared__ int pre[MASW_MAX_BATCH + 1], s_kv[MASW_MAX_BATCH], s_n[MASW_MAX_BATCH], s_r0[MASW_MAX_BATCH];
    const int tid = threadIdx.x, b = blockIdx.x / p.c.Hkv, h = blockIdx.x % p.c.Hkv, G = p.G;
    const int total = make_line<128>(p, pre, s_kv, s_n, s_r0, false);
    const int per = (pre[b + 1] - pre[b]) / p.c.Hkv, T0 = pre[b] + h * per, T1 = T0 + per, nq = s_n[b] * G;
    pdl_wait();
    pdl_trigger();
    if (per == 0) return;
    const int c0 = tile_owner(T0, total, n_cta), c1 = tile_owner(T1 - 1, total, n_cta);
    if (c0 == c1) return;
    for (int r = blockIdx.y * 4; r < imin(nq, (int)blockIdx.y * 4 + 4); ++r) {
        float M = -INFINITY, l = 0.f, o = 0.f;
        for (int c8 = c0; c8 <= c1; c8 += 8) {
            float pm[8], pl[8], po[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = c8 + k, f = first_tile(c, total, n_cta);
                pm[k] = -INFINITY;
                if (c <= c1 && f < first_tile(c + 1, total, n_cta)) {
                    const float* part = p.part + ((size_t)c * 2 + (T0 <= f ? 0 : 1)) * kRowsMax * (D + 2);
                    pm[k] = __ldcg(part + kRowsMax * D + r);
                    pl[k] = __ldcg(part + kRowsMax * (D + 1) + r);
                    po[k] = __ldcg(part + r * D + tid % D);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (pm[k] == -INFINITY) continue;
                const float nm = fmaxf(M, pm[k]);
                const float w0 = exp2f(M - nm), w1 = exp2f(pm[k] - nm);
                l = l * w0 + pl[k] * w1;
                o = o * w0 + po[k] * w1;
                M = nm;
            }
        }
        const size_t row = (size_t)(s_r0[b] + r / G) * p.Hq + h * G + r % G;
        if (tid < D) store_out(p, row * D + tid, l == 0.f ? 0.f : o / l);
        if (tid == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.6931471805599453f;
    }
}

template <bool E4, int D, int NP>
cudaError_t launch(const PagedAttnParams& p, int n_cta, cudaStream_t st) {
    using C = Cfg<E4, D, NP>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(rows_kernel<E4, D, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_release);
    }
    e = masw_launch(rows_kernel<E4, D, NP>, dim3(n_cta), dim3(kThreads), C::kSmem, st, 1, p);
    if (e != cudaSuccess) return e;
    const int nq = p.max_rows * p.G;
    return masw_launch(rows_merge_kernel<D>, dim3(p.c.B * p.c.Hkv, (nq + 3) / 4), dim3(128), 0, st, 1, p, n_cta);
}

}  // namespace rows

cudaError_t launch_paged_rows(const PagedAttnParams& p, int n_cta, cudaStream_t st) {
    const int nq = p.max_rows * p.G;
    auto pick = [&](auto e4, auto d) {
        constexpr bool E4 = decltype(e4)::value;
        constexpr int D = decltype(d)::value;
        if (nq <= 8) return rows::launch<E4, D, 8>(p, n_cta, st);
        if (nq <= 16) return rows::launch<E4, D, 16>(p, n_cta, st);
        return rows::launch<E4, D, 32>(p, n_cta, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.c.k_scale) return p.c.D == 64 ? pick(std::true_type{}, D64{}) : pick(std::true_type{}, D128{});
    return p.c.D == 64 ? pick(std::false_type{}, D64{}) : pick(std::false_type{}, D128{});
}

}  // namespace masw
