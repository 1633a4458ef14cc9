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
//     largest), and so are the weights (p1 + p2 / 16, off by at most 2^-9, half of
//     what rounding them to bf16 would cost): the terms lie side by side in N, so a
//     tile of K or V is read by the tensor core once for both.  The scale of a key's
//     page multiplies its scores; the scale of its value's page enters the
//     exponent, 2^(s + log2 scale - reference), and the sum takes it out again;
//   * bf16 pages: weights as two bf16 terms (2^-17).
// Rows behind the end of a sequence never count: their scores are masked, and
// their V rows are zeroed in shared memory (0 x NaN is NaN in a matrix product).
//
// Measured: decode of 8 sequences at 32K, 24 query and 8 kv heads of 128, e4m3: 87 us
// (6.2 TB/s); 32 sequences of 4K to 16K, 32 query heads, bf16: 211 us (6.7 TB/s, the rate
// of a copy); verify, 6 rows of 4 sequences at 32K, e4m3: 62 us (4.3 TB/s: the softmax
// of 24 rows, not the stream).  The smallest calls (one sequence at 4K: 11 us) are a chain
// of latencies: launch, lengths, page ids, scales, pages, scores, merge.
//
// Warps 0-3 and 4-7: two softmax groups that take the tiles in turn, each with its
// own S, P, O, sums and reference (a tile's chain of barriers, votes and TMEM
// loads is ~1000 cycles long whatever the work in it; one group alone left half of
// the stream's bandwidth unused); the first group joins the two at a pair's end.
// Warp 8 issues S; 9 issues O and loads and splits Q for the next pair; 10 looks up
// pages and scales and loads K, 11 loads V (one warp for both spent 1750 cycles a
// tile on it, more than the 1400 that its bytes take).  Hand-offs are mbarriers;
// every wait is bounded.
#include "masw_paged_attn.cuh"

namespace masw {
namespace rows {

using namespace tc;

constexpr int kThreads = 384;
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
    static constexpr int kSN = E4 ? 2 * NP : (NP + 15) / 16 * 16;            // columns of S^T
    static constexpr int kPN = 2 * NP;                                       // columns of P^T and O^T: two terms
    static constexpr uint32_t kPBuf = kTile * kPN * kES;
    static constexpr uint32_t kQBuf = kSN * kRB;
    static constexpr bool kWide = !E4 && D == 128;              // 32 KB tiles: three stages
    static constexpr int kKS = kWide ? 3 : (kRB == 128 ? 5 : 8);              // K stages
    static constexpr int kVS = kWide && NP > 16 ? 2 : kKS;                    // V stages
    static constexpr int kQBufs = kWide && NP > 16 ? 1 : 2;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKS * kTileB;
    static constexpr uint32_t kOffP = kOffV + kVS * kTileB;
    static constexpr uint32_t kOffQ = kOffP + 2 * kPBuf;
    static constexpr uint32_t kOffQRaw = kOffQ + kQBufs * kQBuf;              // bf16 rows before the split
    static constexpr uint32_t kOffSeq = kOffQRaw + (E4 || kQBufs == 1 ? NP * D * 2 : 0);   // pre[B + 1], kv, n, r0
    static constexpr uint32_t kOffMeta = kOffSeq + 4 * (4 * MASW_MAX_BATCH + 4);
    static constexpr uint32_t kOffStats = kOffMeta + (E4 ? kMeta * 8 * 16 : 0);
    // floats of a group: row maxima [4][NP] of its warps, references [NP], factors
    // [NP], and published at a piece's end: row sums [4][NP] and references [NP];
    // then the joined weights of both groups [2][NP] and the rows' places [NP]
    static constexpr int kRef = 4 * NP, kFac = 5 * NP, kSums = 6 * NP, kOut = 10 * NP, kStats = 11 * NP;
    static constexpr int kFin = 2 * kStats, kRow = kFin + 2 * NP, kStatFloats = kRow + NP;
    static constexpr uint32_t kOffQs = kOffStats + kStatFloats * 4;            // scale of Q per buffer, unset rows per group
    static constexpr uint32_t kOffBar = kOffQs + 16;
    // barriers
    static constexpr int kKFull = 0, kKFree = kKS, kVFull = 2 * kKS, kVFree = kVFull + kVS, kMetaBar = kVFree + kVS;
    static constexpr int kSFull = kMetaBar + (E4 ? kMeta : 0), kSFree = kSFull + 2, kPFull = kSFree + 2, kPFree = kPFull + 2;
    static constexpr int kQFull = kPFree + 2, kQFree = kQFull + 2, kStat = kQFree + 2, kOFree = kStat + 1, kDone = kOFree + 1, kBars = kDone + 2;
    static constexpr uint32_t kSmem = kOffBar + 8 * kBars + 16;               // + TMEM address, abort flag
    static constexpr uint32_t kColO = 2 * kSN;
    static constexpr uint32_t kColsUsed = 2 * kSN + 2 * kPN;
    static constexpr uint32_t kCols = kColsUsed <= 64 ? 64 : (kColsUsed <= 128 ? 128 : (kColsUsed <= 256 ? 256 : 512));
    static constexpr uint32_t kType = E4 ? 0 : 1;               // operand type field: e4m3 / bf16
    static constexpr uint32_t kBase = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(kTile >> 4) << 24);
    static constexpr uint32_t kIdescS = kBase | ((uint32_t)(kSN >> 3) << 17);
    static constexpr uint32_t kIdescO = kBase | (1u << 15) | (1u << 16) | ((uint32_t)(kPN >> 3) << 17);
    // the exponent's reference lies this far below the largest score, and may be
    // exceeded by 2^8: e4m3 weights reach 256 (of 448)
    static constexpr float kHead = E4 ? 6.f : 0.f;
    static_assert(kSmem + 1024 <= 232448, "shared memory");
    static_assert(kKS + 2 < kMeta, "scales would be overwritten");
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

__device__ __forceinline__ bool bar_or(int group, bool x) {   // vote over a group's 128 threads
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)x), "r"(1 + group)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_group(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }

// The softmax groups need more registers than the launch gives a thread when they
// hold over 16 rows: 256 x 216 + 128 x 72 = 384 x 168.
template <int NP>
__device__ __forceinline__ void take_registers() {
    if constexpr (NP > 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
}
template <int NP>
__device__ __forceinline__ void give_registers() {
    if constexpr (NP > 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
}

__device__ __forceinline__ float warp_max(float x) {   // in every lane; NaN does not count
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
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
    const uint32_t abort_flag = sb + C::kOffBar + 8 * C::kBars + 4;
    int* pre = reinterpret_cast<int*>(smem + C::kOffSeq);
    int* s_kv = pre + MASW_MAX_BATCH + 1;
    int* s_n = s_kv + MASW_MAX_BATCH;
    int* s_r0 = s_n + MASW_MAX_BATCH;
    float* stats = reinterpret_cast<float*>(smem + C::kOffStats);
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
            mbar_init(bars + i, i >= C::kQFree && i < C::kQFree + 2                             ? 9
                                : (i >= C::kSFree && i < C::kSFree + 2) || (i >= C::kPFull && i < C::kPFull + 2) ||
                                          i == C::kStat || i == C::kOFree
                                      ? 4
                                      : 1);
        st_shared_u32(abort_flag, 0u);
        fence_mbar_init();
    }
    if (tid == 32) {
        tma_prefetch_map(&p.tm_k);
        tma_prefetch_map(&p.tm_v);
    }
    pdl_wait();
    pdl_trigger();
    const Line line = make_line<kThreads>(p, pre, s_kv, s_n, s_r0, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    Walk walk;
    if (const int per_pair = pair_ctas(B * Hkv, line.longest, line.total, gridDim.x)) {
        const int pair = blockIdx.x / per_pair, part = blockIdx.x - pair * per_pair, h = pair % Hkv;
        walk.b = imin(pair / Hkv, B - 1);
        const int nt = pair < B * Hkv ? (pre[walk.b + 1] - pre[walk.b]) / Hkv : 0;
        walk.t = pre[walk.b] + h * nt + part_first(part, nt, per_pair);
        walk.t1 = pre[walk.b] + h * nt + part_first(part + 1, nt, per_pair);
    } else {
        walk.t = first_tile(blockIdx.x, line.total, gridDim.x);
        walk.t1 = first_tile(blockIdx.x + 1, line.total, gridDim.x);
        int lo = 0, hi = B;   // the sequence of the first tile
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= walk.t) lo = mid;
            else hi = mid;
        }
        walk.b = lo;
    }
    auto wait = [&](int bar, int phase) { return wait_bounded(bar_at(bar), (uint32_t)phase & 1u, abort_flag, p.status); };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    bool ok = true;

    // one register change for each whole group of four warps
    if (warp >= 8) {
        give_registers<NP>();
        if (warp == 8) {
            // ---------------- S^T = K Q^T ----------------
            int i = 0, piece = 0;
            while (ok && next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
                const int qb = piece % C::kQBufs;
                ok = all(wait(C::kQFull + qb, piece / C::kQBufs));
                const uint64_t bq = smem_desc(sb + C::kOffQ + qb * C::kQBuf, 128, (C::kRB / 16) * 128, 0);
                for (int j = 0; ok && j < walk.nt; ++j, ++i) {
                    const int st = i % C::kKS, sbuf = i & 1;
                    ok = all(wait(C::kKFull + st, i / C::kKS)) && (i < 2 || all(wait(C::kSFree + sbuf, i / 2 - 1)));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ak = smem_desc(sb + C::kOffK + st * C::kTileB, 16, C::kAtom, C::kSwz);
                    if (elect_one()) {
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
                    __syncwarp();
                }
                ++piece;
            }
            // nothing may arrive on a barrier after the CTA ended
            if (ok && i > 0)
                ok = all(wait(C::kKFree + (i - 1) % C::kKS, (i - 1) / C::kKS)) &&
                     all(wait(C::kQFree + (piece - 1) % C::kQBufs, (piece - 1) / C::kQBufs));
            if (!ok) {   // let the matrix products in flight end before the CTA does
                st_shared_u32(abort_flag, 1u);
                if (elect_one()) umma_commit(bar_at(C::kDone));
                __syncwarp();
                mbar_wait(bars + C::kDone, 0, nullptr);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---------------- O^T += V^T P^T, and Q of the next piece ----------------
            // Q in 16-byte chunks: a row is kLanes of them, a pass kPer rows; every lane
            // splits the chunks that it copied itself.  Loops stay rolled, here and wherever
            // code runs once a piece: fetching instructions for the first time costs more
            // than running them.  The copies of the next piece's
            // rows are issued at a piece's start and finished after its second tile.
            constexpr int kLanes = D / 8, kPer = 32 / kLanes, kPass = NP / kPer;
            const int e0 = (lane % kLanes) * 8, rl = lane / kLanes;
            const uint32_t raw = sb + C::kOffQRaw + (uint32_t)lane * 16u;   // pass s: 512 bytes further
            Walk wq = walk;
            int q_piece = 0;
            // K-major core matrices of 8 rows x 16 bytes, consecutive along the row
            auto at = [&](int row, int byte) {
                return sb + C::kOffQ + (q_piece % C::kQBufs) * C::kQBuf +
                       (uint32_t)((row >> 3) * (C::kRB / 16) * 128 + (byte >> 4) * 128 + (row & 7) * 16 + (byte & 15));
            };
            auto q_free = [&]() {
                return q_piece < C::kQBufs || all(wait(C::kQFree + q_piece % C::kQBufs, q_piece / C::kQBufs - 1));
            };
            auto q_issue = [&]() {
                if (!next_piece(wq, pre, B, Hkv, s_kv, s_n, p.window)) return false;
                // bf16: straight into the operand, once the matrix products that read it are
                // done; with one buffer that is at the end of the piece
                if (!E4 && C::kQBufs > 1) ok = q_free();
                const int nq = s_n[wq.b] * G, r0 = s_r0[wq.b];
                int tok = rl / G, g = rl - tok * G;
#pragma unroll 1
                for (int s = 0; s < kPass; ++s) {
                    const int r = s * kPer + rl;
                    const bool in = r < nq;
                    const __nv_bfloat16* src = p.q + (size_t)(r0 + (in ? tok : 0)) * p.q_stride + (size_t)(wq.h * G + (in ? g : 0)) * D + e0;
                    if (E4 || C::kQBufs == 1) {
                        cp_async16(raw + s * 512, src, in ? 16 : 0);
                    } else {
                        cp_async16(at(r, e0 * 2), src, in ? 16 : 0);
                        if (NP + r < C::kSN) st_shared_v4(at(NP + r, e0 * 2), 0u, 0u, 0u, 0u);
                    }
                    g += kPer;
                    while (g >= G) {
                        g -= G;
                        ++tok;
                    }
                }
                cp_async_commit();
                return true;
            };
            auto q_finish = [&]() {
                cp_async_wait<0>();
                float inv = 1.f;
                if constexpr (E4) {
                    float amax = 0.f;
#pragma unroll 1
                    for (int s = 0; s < kPass; ++s) {
                        const float4 v = ld_shared_v4f(raw + s * 512);
                        float f[8];
                        Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(&v), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(f[e]));
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    inv = 1.f / pow2_scale(amax);
                    ok = ok && q_free();
#pragma unroll 1
                    for (int s = 0; s < kPass; ++s) {
                        const int r = s * kPer + rl;
                        const float4 v = ld_shared_v4f(raw + s * 512);
                        float f[8];
                        Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(&v), f);
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
                        st_shared_v2(at(r, e0), w1[0] | (w1[1] << 16), w1[2] | (w1[3] << 16));
                        st_shared_v2(at(NP + r, e0), w2[0] | (w2[1] << 16), w2[2] | (w2[3] << 16));
                    }
                } else if constexpr (C::kQBufs == 1) {
                    ok = ok && q_free();
#pragma unroll 1
                    for (int s = 0; s < kPass; ++s) {
                        const int r = s * kPer + rl;
                        const float4 v = ld_shared_v4f(raw + s * 512);
                        const uint4 x = *reinterpret_cast<const uint4*>(&v);
                        st_shared_v4(at(r, e0 * 2), x.x, x.y, x.z, x.w);
                        if (NP + r < C::kSN) st_shared_v4(at(NP + r, e0 * 2), 0u, 0u, 0u, 0u);
                    }
                }
                if (!ok) return;
                const int qb = q_piece % C::kQBufs;
                if (lane == 0) qscale[qb] = p.scale_log2 / inv;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kQFull + qb));
                ++q_piece;
            };
            // one operand buffer: it is free only when the piece's own products are done
            constexpr bool kLate = C::kQBufs == 1;
            if (q_issue()) q_finish();
            int i = 0;
            while (ok && next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
                bool pending = q_issue();
                for (int j = 0; ok && j < walk.nt; ++j, ++i) {
                    const int st = i % C::kVS, pb = i & 1;
                    ok = all(wait(C::kPFull + pb, i / 2)) && all(wait(C::kVFull + st, i / C::kVS));
                    if (!ok) break;
                    tc_fence_after();
                    // head_dim 64: the second half of the 128 M rows repeats the first
                    // (a leading offset of 0); head_dim 128 in bf16: the second panel
                    const uint64_t av = smem_desc(sb + C::kOffV + st * C::kTileB, C::kPanels == 2 ? C::kPanel : 0, C::kAtom, C::kSwz);
                    const uint64_t bp = smem_desc(sb + C::kOffP + pb * C::kPBuf, 128, 2048, 0);
                    constexpr int kKeys = 32 / C::kES;   // keys of one matrix instruction
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kTile / kKeys; ++kk) {
                            const uint64_t a = av + (uint64_t)((kk * kKeys * C::kPB) >> 4);
                            const uint64_t b = bp + (uint64_t)((kk * kKeys * 16) >> 4);
                            if (E4) umma_f8(tmem + C::kColO + pb * C::kPN, a, b, C::kIdescO, j > 1 || kk > 0);
                            else umma_bf16(tmem + C::kColO + pb * C::kPN, a, b, C::kIdescO, j > 1 || kk > 0);
                        }
                        umma_commit(bar_at(C::kPFree + pb));
                        umma_commit(bar_at(C::kVFree + st));
                    }
                    __syncwarp();
                    if (pending && j + 1 == (kLate ? walk.nt : imin(2, walk.nt))) {
                        q_finish();
                        pending = false;
                    }
                }
            }
            // nothing may arrive on a barrier after the CTA ended
            if (ok && i > 0) ok = all(wait(C::kVFree + (i - 1) % C::kVS, (i - 1) / C::kVS));
            if (!ok) {
                st_shared_u32(abort_flag, 1u);
                cp_async_wait<0>();
                if (elect_one()) umma_commit(bar_at(C::kDone + 1));
                __syncwarp();
                mbar_wait(bars + C::kDone + 1, 0, nullptr);
            }
            __syncwarp();
        } else {
            // ---------------- page ids and TMA: warp 10 K and the scales, warp 11 V ----------------
            // A lane holds the page of one box (at most 128 rows of a page); a batch
            // is up to 32 boxes of a piece.  Page ids are loaded two batches ahead, scales
            // one.
            const bool is_v = warp == 11;
            const int stages = is_v ? C::kVS : C::kKS, full = is_v ? C::kVFull : C::kKFull, freed = is_v ? C::kVFree : C::kKFree;
            const uint32_t ring = sb + (is_v ? C::kOffV : C::kOffK);
            const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
            const bool scales = E4 && !is_v;
            const int box = imin(c.P, kTile), bpt = kTile / box, bt = 32 / bpt;   // boxes a tile, tiles a batch
            int left = 0, at = 0;            // tiles of the piece not yet in a batch, and the first of them
            struct Batch { int h, tile, nt, pid, lo, hi; bool in; float ks, vs; };   // boxes [lo, hi) hold visible keys
            auto next_batch = [&](Batch& x) {
                x.nt = 0;
                x.in = false;
                if (left == 0) {
                    if (!next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) return;
                    left = walk.nt;
                    at = walk.tile;
                }
                x.h = walk.h;
                x.tile = at;
                x.nt = imin(left, bt);
                at += x.nt;
                left -= x.nt;
                const TileRange r = tile_range(s_n[walk.b], s_kv[walk.b], p.window);
                const int key0 = x.tile * kTile;
                x.lo = imax(0, r.lo / c.P * c.P - key0) / box;   // pages wholly before the first visible key are left out
                x.hi = imin(x.nt * bpt, (r.hi - key0 + box - 1) / box);
                x.in = lane >= x.lo && lane < x.hi;
                x.pid = x.in ? __ldg(c.table + (size_t)walk.b * c.table_stride + (key0 + lane * box) / c.P) : 0;
            };
            auto check_and_scale = [&](Batch& x) {
                if (x.in && (x.pid < 0 || x.pid >= c.n_pages)) {
                    if (p.status) atomicExch(p.status, MASW_EINVAL);
                    x.pid = 0;
                }
                x.ks = x.vs = 1.f;
                if (scales && x.in) {
                    x.ks = __ldg(c.k_scale + (size_t)x.pid * Hkv + x.h);
                    x.vs = __ldg(c.v_scale + (size_t)x.pid * Hkv + x.h);
                }
            };
            Batch cur, nxt;
            int i = 0, st = 0, turn = 0;     // tile, its stage, and how often the ring went round
            next_batch(cur);
            next_batch(nxt);
            check_and_scale(cur);
            while (ok && cur.nt > 0) {
                check_and_scale(nxt);
                Batch nn;
                next_batch(nn);
                for (int j = 0; j < cur.nt; ++j, ++i) {
                    const int b0 = imax(cur.lo, j * bpt), b1 = imin(cur.hi, (j + 1) * bpt);   // the tile's boxes
                    if (turn > 0) ok = all(wait(freed + st, turn - 1));
                    if (!ok) break;
                    if (elect_one()) mbar_expect_tx_at(bar_at(full + st), (uint32_t)(imax(0, b1 - b0) * box * C::kRB));
                    __syncwarp();
                    // the whole warp walks the boxes, one lane issues
                    for (int q = b0; q < b1; ++q) {
                        const int pid = __shfl_sync(0xffffffffu, cur.pid, q);
                        const int row = (cur.tile * kTile + q * box) & (c.P - 1);
                        const uint32_t dst = ring + st * C::kTileB + (uint32_t)((q - j * bpt) * box * C::kPB);
                        if (elect_one()) {
#pragma unroll
                            for (int pn = 0; pn < C::kPanels; ++pn)
                                tma_load_4d(dst + pn * C::kPanel, map, pn * C::kPB / C::kES, row, cur.h, pid, bar_at(full + st));
                        }
                    }
                    __syncwarp();
                    if (scales) {   // behind the copies, which need not wait for them
                        if (lane / bpt == j)
                            st_shared_v4(sb + C::kOffMeta + (uint32_t)((i % kMeta) * 8 + lane % bpt) * 16u, __float_as_uint(cur.ks),
                                         __float_as_uint(cur.vs == 1.f ? 0.f : __log2f(cur.vs)), __float_as_uint(__frcp_rn(cur.vs)), 0u);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_at(C::kMetaBar + i % kMeta));
                    }
                    if (++st == stages) {
                        st = 0;
                        ++turn;
                    }
                }
                cur = nxt;
                nxt = nn;
            }
            // after a wait gave up, and at the end: no copy may be in flight when the CTA ends
            if (!ok) st_shared_u32(abort_flag, 1u);
            for (int k = imax(0, i - stages); k < i; ++k)
                mbar_wait(bars + full + k % stages, (uint32_t)(k / stages) & 1u, nullptr);
            __syncwarp();
        }
    } else {
        take_registers<NP>();
        // ---------------- softmax: thread wt of a group owns key wt of the group's tiles ----------------
        // After a wait gave up these warps go on to the end of their tiles (every
        // later wait returns at once), so that they meet at their barriers.
        const int group = warp >> 2, wt = tid & 127, gw = warp & 3;
        const uint32_t lane_off = (uint32_t)(gw * 32) << 16;
        const uint32_t t_s = tmem + group * C::kSN + lane_off;
        const uint32_t t_o = tmem + C::kColO + lane_off;             // group 0's; group 1's kPN columns further
        const uint32_t t_own = t_o + group * C::kPN;
        float* own = stats + group * C::kStats;
        const uint32_t own_a = smem_u32(own);
        uint32_t* unset_word = reinterpret_cast<uint32_t*>(qscale) + 2 + group;
        int i0 = 0, piece = 0;
        bool first = true;
        while (next_piece(walk, pre, B, Hkv, s_kv, s_n, p.window)) {
            const int b = walk.b, n = s_n[b], kv = s_kv[b], nq = n * G, q_pos = kv - n;
            const TileRange range = tile_range(n, kv, p.window);
            const int qb = piece % C::kQBufs;
            // keys that every row sees: [all_lo, all_hi)
            const int all_hi = q_pos + 1, all_lo = p.window > 0 ? imax(0, kv - p.window) : 0;
            // rows without a reference yet, because they have seen no key (the same in
            // every thread of the group)
            uint32_t unset = nq == 32 ? 0xffffffffu : (1u << nq) - 1u;
            float l[NP];
#pragma unroll
            for (int r = 0; r < NP; ++r) l[r] = 0.f;
            if (wt < NP) own[C::kRef + wt] = 0.f;
            bar_group(group);
            ok &= wait(C::kQFull + qb, piece / C::kQBufs);
            const float qs = qscale[qb];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_at(C::kQFree + qb));
            bool o_free = group == 0 || piece == 0;   // group 0 has read this group's O and sums of the last piece
            for (int j = (i0 ^ group) & 1; j < walk.nt; j += 2) {
                const int i = i0 + j, turn = i >> 1;
                const int tile0 = (walk.tile + j) * kTile, key = tile0 + wt;
                const bool masked = tile0 < all_lo || tile0 + kTile > all_hi;
                const bool seen = key >= range.lo && key < range.hi;   // by some row
                uint32_t see = 0xffffffffu;                            // by which rows
                float ks = qs, lvs = 0.f, ivs = 1.f;
                if (E4) {
                    ok &= wait(C::kMetaBar + i % kMeta, i / kMeta);
                    const float4 mt = ld_shared_v4f(sb + C::kOffMeta + (uint32_t)((i % kMeta) * 8 + (c.P >= kTile ? 0 : wt / c.P)) * 16u);
                    ks *= mt.x;
                    lvs = mt.y;
                    ivs = mt.z;
                }
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
                    const int st = i % C::kVS;
                    // A wait tells a phase only from its neighbours, so the stage's tile before
                    // has to have landed: with four stages it has (this group's last but one
                    // product is done), with fewer once the group's last one is.
                    if (C::kVS < 4 && turn > 0) ok &= wait(C::kPFree + group, turn - 1);
                    ok &= wait(C::kVFull + st, i / C::kVS);
                    if (!seen) {
#pragma unroll
                        for (int pn = 0; pn < C::kPanels; ++pn)
#pragma unroll
                            for (int q = 0; q < C::kPB / 16; ++q)
                                st_shared_v4(sb + C::kOffV + st * C::kTileB + pn * C::kPanel + wt * C::kPB + q * 16, 0u, 0u, 0u, 0u);
                    }
                }
                ok &= wait(C::kSFull + group, turn);
                __syncwarp();
                tc_fence_after();
                // a: this key's scores of all rows in the log2 domain (the V scale with
                // them) relative to the rows' references; -inf where a row does not see
                // the key.  A reference moves when a score exceeds it by more than 2^8,
                // and O and the sums shrink with it; then a is computed anew.
                float a[NP];
                bool p_free = turn == 0;
#pragma unroll 1
                for (;;) {
                    {
                        uint32_t sv[E4 ? 2 * NP : NP];
                        tmem_ld_cols<E4 ? 2 * NP : NP>(t_s, sv);
                        tmem_wait_ld();
#pragma unroll
                        for (int r = 0; r < NP; r += 4) {
                            const float4 m = ld_shared_v4f(own_a + (C::kRef + r) * 4);
                            const float mr[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = E4 ? fmaf(__uint_as_float(sv[NP + r + e]), 0.0625f, __uint_as_float(sv[r + e]))
                                                   : __uint_as_float(sv[r + e]);
                                a[r + e] = fmaf(x, ks, lvs - mr[e]);
                            }
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int r = 0; r < NP; ++r) a[r] = (see >> r) & 1u ? a[r] : -INFINITY;
                    }
                    float mx = a[0];
#pragma unroll
                    for (int r = 1; r < NP; ++r) mx = fmaxf(mx, a[r]);
                    bool move = mx > 8.f;
                    if (unset) {
#pragma unroll
                        for (int r = 0; r < NP; ++r) move = move || (((unset >> r) & 1u) && a[r] > -3e38f);
                    }
                    if (!bar_or(group, move)) break;
#pragma unroll
                    for (int r = 0; r < NP; ++r) {
                        const float s = warp_max(a[r]);
                        if (lane == 0) own[gw * NP + r] = s;
                    }
                    bar_group(group);
                    if (gw == 0) {
                        float top = -INFINITY;
                        if (lane < NP) {
                            top = fmaxf(fmaxf(own[lane], own[NP + lane]), fmaxf(own[2 * NP + lane], own[3 * NP + lane]));
                            const bool fresh = (unset >> lane) & 1u;
                            const float up = fresh ? (top > -3e38f ? top - C::kHead : 0.f) : fmaxf(0.f, top - C::kHead);
                            own[C::kRef + lane] += up;
                            own[C::kFac + lane] = fresh ? 1.f : ex2_approx(-up);   // what the sums and O shrink by
                        }
                        const uint32_t seen_now = __ballot_sync(0xffffffffu, top > -3e38f);
                        if (lane == 0) *unset_word = unset & ~seen_now;
                    }
                    bar_group(group);
                    unset = *reinterpret_cast<volatile uint32_t*>(unset_word);
#pragma unroll
                    for (int r = 0; r < NP; r += 4) {
                        const float4 f = ld_shared_v4f(own_a + (C::kFac + r) * 4);
                        l[r] *= f.x;
                        l[r + 1] *= f.y;
                        l[r + 2] *= f.z;
                        l[r + 3] *= f.w;
                    }
                    if (j > 1) {
                        // O holds the group's earlier tiles of the piece once the last product is done
                        if (!p_free) ok &= wait(C::kPFree + group, turn - 1);
                        p_free = true;
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < C::kPN; q += 8) {
                            uint32_t ov[8];
                            tmem_ld8(t_own + q, ov);
                            tmem_wait_ld();
                            const uint32_t fa = own_a + (C::kFac + q % NP) * 4;
                            const float4 f0 = ld_shared_v4f(fa), f1 = ld_shared_v4f(fa + 16);
                            const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f[e]);
                            tmem_st8(t_own + q, ov);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kSFree + group));
#pragma unroll
                for (int r = 0; r < NP; ++r) {
                    a[r] = ex2_approx(a[r]);
                    l[r] = fmaf(a[r], ivs, l[r]);
                }
                if (!p_free) ok &= wait(C::kPFree + group, turn - 1);
                // this key's weights of all rows, first terms then second ones, in
                // 16-byte chunks of core matrices (8 keys x 16 bytes)
                const uint32_t pw = sb + C::kOffP + group * C::kPBuf + (uint32_t)((wt >> 3) * 128 + (wt & 7) * 16);
                uint32_t w[C::kPN * C::kES / 4];
                if constexpr (E4) {
#pragma unroll
                    for (int r = 0; r < NP; r += 4) {
                        const uint32_t h0 = cvt_f16x2(a[r], a[r + 1]), h1 = cvt_f16x2(a[r + 2], a[r + 3]);
                        w[r / 4] = e4m3x4(h0, h1);
                        uint32_t e0, e1;
                        e4m3x4_to_f16x2(w[r / 4], e0, e1);
                        w[NP / 4 + r / 4] = e4m3x4(rest16(h0, e0), rest16(h1, e1));
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < NP; r += 2) {
                        w[r / 2] = pack_bf16(a[r], a[r + 1]);
                        w[NP / 2 + r / 2] = pack_bf16(a[r] - bf16lo(w[r / 2]), a[r + 1] - bf16hi(w[r / 2]));
                    }
                }
#pragma unroll
                for (int q = 0; q < C::kPN * C::kES / 16; ++q)
                    st_shared_v4(pw + q * 2048, w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                if (!o_free) {
                    ok &= wait(C::kOFree, piece - 1);
                    o_free = true;
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kPFull + group));
            }
            // the piece's sums over the group's keys: eight rows at a time, a butterfly
            // that halves the rows with every step; lane 4 k ends with row k's sum
            if (!o_free) ok &= wait(C::kOFree, piece - 1);
#pragma unroll
            for (int q = 0; q < NP; q += 8) {
#pragma unroll
                for (int h = 4; h >= 1; h >>= 1) {
                    const bool up = lane & (4 * h);
#pragma unroll
                    for (int e = 0; e < h; ++e) {
                        const float keep = up ? l[q + h + e] : l[q + e], give = up ? l[q + e] : l[q + h + e];
                        l[q + e] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * h);
                    }
                }
                l[q] += __shfl_xor_sync(0xffffffffu, l[q], 2);
                l[q] += __shfl_xor_sync(0xffffffffu, l[q], 1);
                if ((lane & 3) == 0) own[C::kSums + gw * NP + q + (lane >> 2)] = l[q];
            }
            if (wt < NP) own[C::kOut + wt] = (unset >> wt) & 1u ? -1e30f : own[C::kRef + wt];
            const int i1 = i0 + walk.nt;
            if (group == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kStat));
            } else {
                // join the two groups: thread r the sums of row r, then thread d the
                // outputs of element d
                const bool had0 = walk.nt > 1 || !(i0 & 1), had1 = walk.nt > 1 || (i0 & 1);
                float* part = p.part + ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * kRowsMax * (D + 2);
                bar_group(group);
                ok &= wait(C::kStat, piece);
                if (wt < NP) {
                    const int r = wt;
                    const float* s0 = stats + r;
                    const float* s1 = s0 + C::kStats;
                    const float m0 = s0[C::kOut], m1 = s1[C::kOut], m = fmaxf(m0, m1);
                    float w0 = ex2_approx(m0 - m), w1 = ex2_approx(m1 - m);
                    const float sum = (s0[C::kSums] + s0[C::kSums + NP] + s0[C::kSums + 2 * NP] + s0[C::kSums + 3 * NP]) * w0 +
                                      (s1[C::kSums] + s1[C::kSums + NP] + s1[C::kSums + 2 * NP] + s1[C::kSums + 3 * NP]) * w1;
                    int place = r;
                    if (walk.whole) {
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        w0 *= inv;
                        w1 *= inv;
                        place = (s_r0[b] + r / G) * p.Hq + walk.h * G + r % G;
                        if (r < nq && p.lse) p.lse[place] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
                    } else if (r < nq) {
                        __stcg(part + kRowsMax * D + r, sum == 0.f ? -INFINITY : m);
                        __stcg(part + kRowsMax * (D + 1) + r, sum);
                    }
                    stats[C::kFin + r] = w0;
                    stats[C::kFin + NP + r] = w1;
                    reinterpret_cast<int*>(stats)[C::kRow + r] = place;
                }
                if (had0) ok &= wait(C::kPFree, (i1 - 1) >> 1);
                if (had1) ok &= wait(C::kPFree + 1, (i1 - 2) >> 1);
                bar_group(group);
                tc_fence_after();
                const bool f32 = p.o_f32 || !walk.whole;
                float* fdst = walk.whole ? reinterpret_cast<float*>(p.o) : part;
#pragma unroll 1
                for (int q = 0; q < nq; q += 8) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!(g ? had1 : had0)) continue;
                        uint32_t u[8], v[8];
                        tmem_ld8(t_o + g * C::kPN + q, u);
                        tmem_ld8(t_o + g * C::kPN + NP + q, v);
                        const uint32_t wa = smem_u32(stats + C::kFin + g * NP + q);
                        const float4 w0 = ld_shared_v4f(wa), w1 = ld_shared_v4f(wa + 16);
                        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = fmaf(fmaf(__uint_as_float(v[e]), E4 ? 0.0625f : 1.f, __uint_as_float(u[e])), w[e], o[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (q + e < nq && wt < D) {
                            const size_t at = (size_t)reinterpret_cast<const int*>(stats)[C::kRow + q + e] * D + wt;
                            if (f32) __stcg(fdst + at, o[e]);
                            else reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(o[e]);
                        }
                    }
                }
                tc_fence_before();
                bar_group(group);   // the joined weights were read
                if (lane == 0) mbar_arrive(bar_at(C::kOFree));
            }
            i0 = i1;
            first = false;
            ++piece;
        }
        if (!ok) st_shared_u32(abort_flag, 1u);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
    }
}

// Joins the pieces of the pairs that were cut.  CTA (pair, rows): D / 4 threads own
// a row, four output elements each.
constexpr int kMergeThreads = 256, kAtOnce = 8;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) rows_merge_kernel(const __grid_constant__ PagedAttnParams p, int n_cta) {
    __shared__ int pre[MASW_MAX_BATCH + 1], s_kv[MASW_MAX_BATCH], s_n[MASW_MAX_BATCH], s_r0[MASW_MAX_BATCH];
    const int pair = blockIdx.x, b = pair / p.c.Hkv, h = pair % p.c.Hkv, G = p.G;
    const int r = blockIdx.y * (kMergeThreads * 4 / D) + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
    const Line line = make_line<kMergeThreads>(p, pre, s_kv, s_n, s_r0, false);
    const int nt = (pre[b + 1] - pre[b]) / p.c.Hkv, T0 = pre[b] + h * nt, nq = s_n[b] * G;
    const int per_pair = pair_ctas(p.c.B * p.c.Hkv, line.longest, line.total, n_cta);
    int c0 = 0, c1 = 0;
    if (nt > 0) {
        c0 = per_pair ? pair * per_pair : tile_owner(T0, line.total, n_cta);
        c1 = per_pair ? c0 + imin(nt, per_pair) - 1 : tile_owner(T0 + nt - 1, line.total, n_cta);
    }
    pdl_wait();
    pdl_trigger();
    if (c0 == c1 || r >= nq) return;
    float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c8 = c0; c8 <= c1; c8 += kAtOnce) {
        float pm[kAtOnce], pl[kAtOnce];
        float4 po[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            pm[k] = -INFINITY;
            pl[k] = 0.f;
            po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c8 + k <= c1) {
                const int c = c8 + k;
                const int slot = per_pair || T0 <= first_tile(c, line.total, n_cta) ? 0 : 1;
                const float* part = p.part + ((size_t)c * 2 + slot) * kRowsMax * (D + 2);
                pm[k] = __ldcg(part + kRowsMax * D + r);
                pl[k] = __ldcg(part + kRowsMax * (D + 1) + r);
                po[k] = __ldcg(reinterpret_cast<const float4*>(part + r * D + d));
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, pm[k]);
        if (top == -INFINITY) continue;
        const float w = exp2f(M - top);
        l *= w;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= w;
        M = top;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float wk = exp2f(pm[k] - M);
            l = fmaf(pl[k], wk, l);
            if (pm[k] == -INFINITY) continue;
            o[0] = fmaf(po[k].x, wk, o[0]);
            o[1] = fmaf(po[k].y, wk, o[1]);
            o[2] = fmaf(po[k].z, wk, o[2]);
            o[3] = fmaf(po[k].w, wk, o[3]);
        }
    }
    const size_t row = (size_t)(s_r0[b] + r / G) * p.Hq + h * G + r % G;
#pragma unroll
    for (int e = 0; e < 4; ++e) store_out(p, row * D + d + e, l == 0.f ? 0.f : o[e] / l);
    if (d == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.6931471805599453f;
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
    constexpr int kRows = kMergeThreads * 4 / D;
    return masw_launch(rows_merge_kernel<D>, dim3(p.c.B * p.c.Hkv, (p.max_rows * p.G + kRows - 1) / kRows), dim3(kMergeThreads), 0,
                       st, 1, p, n_cta);
}

}  // namespace rows

cudaError_t launch_paged_rows(const PagedAttnParams& p, int n_cta, cudaStream_t st) {
    const int nq = p.max_rows * p.G;
    auto pick = [&](auto e4, auto d) {
        constexpr bool E4 = decltype(e4)::value;
        constexpr int D = decltype(d)::value;
        if (nq <= 8) return rows::launch<E4, D, 8>(p, n_cta, st);
        if (nq <= 16) return rows::launch<E4, D, 16>(p, n_cta, st);
        if (nq <= 24) return rows::launch<E4, D, 24>(p, n_cta, st);
        return rows::launch<E4, D, 32>(p, n_cta, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.c.k_scale) return p.c.D == 64 ? pick(std::true_type{}, D64{}) : pick(std::true_type{}, D128{});
    return p.c.D == 64 ? pick(std::false_type{}, D64{}) : pick(std::false_type{}, D128{});
}

}  // namespace masw
