// Attention of many query rows a sequence over a paged cache (chunks of a prompt,
// longer query blocks): 256 rows (query token x query head of the group) of a
// (sequence, kv head) pair a CTA.
//
// A dense contraction, bound by the tensor cores once the rows share enough of
// the cache: 4 D flops a row and visible key.  Two tiles of 128 rows go through
// the keys together, 128 keys at a time, in turn: while the softmax of one tile
// runs, the tensor cores work on the other one.  Per tile S = Q K^T (M = 128 rows,
// N = 128 keys) and O += P V (N = head_dim) accumulate in tensor memory; two
// threads own a row, one for each half of the keys.  (One thread a row spent 2000
// cycles on a tile, and the tensor cores waited for it.)  P replaces S in tensor memory and is
// the A operand of P V from there; matrix instructions of one thread run in the
// order of their issue, so the next S follows the P V that reads P.
// e4m3 pages: K enters as it is, against Q as two e4m3 terms (twice the instructions
// at twice the bf16 rate); V is widened to fp16 in shared memory, which is exact,
// once for both tiles, so that the weights enter as fp16 (off by at most 2^-11):
// splitting the weights into e4m3 terms instead took a third of the softmax's
// instructions.  The scales of a page multiply its columns of S and enter the
// exponent as in the few-rows kernel.  bf16 pages: weights rounded to bf16 (2^-8 at
// most; the outputs are means over many of them).
//
// Warps 0-7 and 8-15: softmax of the two tiles; 16 issues the matrix products of
// the tiles in turn, all of a tile's at once: P V and the next S of one tile run
// while the other one's softmax does (with an issuing warp a tile the products of
// both interleaved, ended together, and left the tensor cores idle during both
// softmaxes); 17 watches K and V for it, so that one barrier stands before a step.  18: page ids,
// scales and K; 19: page ids and V; 20-23 widen V and clear the rows that no query
// sees.  A long cache under few rows is cut into splits, whose partial results a second
// kernel joins.
//
// Measured: a 2K chunk at 32K, 32 query and 8 kv heads of 128, e4m3: 765 us (1393
// TFLOP/s); prompts of up to 4K, 24 query heads, bf16: 240 us (850 TFLOP/s: a CTA's start
// and end, ~9 us, against a mean of 8 tiles of keys).  A tile of keys for both tiles
// of rows takes ~2.9K cycles, of which the matrix products are ~2.1K.
#include "masw_paged_attn.cuh"

namespace masw {
namespace tile {

using namespace tc;

constexpr int kThreads = 768;
constexpr int kMeta = 8;
// Weights may reach 2^14 (fp16 ends at 2^16; what lies 2^-38 below the largest is
// lost): a row's reference then hardly ever moves after its first tile, and moving
// it stalls the tile for ~2000 cycles.
constexpr float kSlack = 14.f;

template <bool E4, int D>
struct Cfg {
    static constexpr int kES = E4 ? 1 : 2;
    static constexpr int kRB = D * kES;
    static constexpr int kPanels = kRB > 128 ? 2 : 1;
    static constexpr int kPB = kRB / kPanels;
    static constexpr uint32_t kPanel = kTile * kPB;
    static constexpr uint32_t kTileB = kTile * kRB;
    static constexpr uint32_t kSwz = kPB == 128 ? 2 : 4;
    static constexpr uint32_t kAtom = 8 * kPB;
    static constexpr int kTerms = E4 ? 2 : 1;                   // of Q
    // stages of K and V (a load takes ~3000 cycles, two tiles' worth; e4m3's V stages
    // are free once widened), and buffers of V as the products read it (bf16: the
    // stages)
    static constexpr int kKS = D == 64 ? 4 : 3, kVS = D == 64 ? 4 : (E4 ? 3 : 2);
    static constexpr int kWS = E4 ? 2 : kVS;
    // V as the products read it, 2 bytes an element: panels of 64 elements
    static constexpr int kWPanels = D / 64;
    static constexpr uint32_t kWPanel = kTile * 128;
    static constexpr uint32_t kWideB = kWPanels * kWPanel;
    static constexpr uint32_t kOffQ = 0;                        // [2 tiles][terms]; bf16: panels of 64 elements
    static constexpr uint32_t kOffK = kOffQ + 2 * kTerms * kTileB;
    static constexpr uint32_t kOffV = kOffK + kKS * kTileB;
    static constexpr uint32_t kOffW = E4 ? kOffV + kVS * kTileB : kOffV;
    // e4m3: the bf16 rows of Q land where V will be widened
    static constexpr uint32_t kOffLand = E4 ? kOffW : kOffQ;
    static constexpr uint32_t kOffMeta = kOffW + kWS * kWideB;
    static constexpr uint32_t kOffRow = kOffMeta + (E4 ? kMeta * 8 * 16 : 0);   // a float a row of both tiles; the second's references
    static constexpr uint32_t kOffBar = kOffRow + 3 * kTile * 4;
    static constexpr int kKFull = 0, kKFree = kKS, kVFull = 2 * kKS, kVFree = kVFull + kVS, kWFull = kVFree + kVS, kWFree = kWFull + kWS, kMetaBar = kWFree + kWS;
    static constexpr int kSFull = kMetaBar + (E4 ? kMeta : 0), kGo = kSFull + 2, kOFull = kGo + 2;   // kGo: all that a step of a tile needs
    static constexpr int kQLand = kOFull + 2;
    static constexpr int kDone = kQLand + 1, kBars = kDone + 1;
    static constexpr uint32_t kSmem = kOffBar + 8 * kBars + 16;
    static constexpr uint32_t kColS = 0, kColO = 256;           // per tile 128 columns of S (or P) and of O
    static constexpr uint32_t kType = E4 ? 0 : 1;
    static constexpr uint32_t kBase = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(kTile >> 4) << 24);
    static constexpr uint32_t kIdescS = kBase | ((uint32_t)(kTile >> 3) << 17);
    static constexpr uint32_t kIdescO = (1u << 4) | ((E4 ? 0u : 1u) << 7) | ((E4 ? 0u : 1u) << 10) | ((uint32_t)(kTile >> 4) << 24) |
                                        (1u << 16) | ((uint32_t)(D >> 3) << 17);   // fp16 or bf16
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kKS + 1 < kMeta, "scales would be overwritten");
};

// Barrier of the two warps (64 threads) that hold the same 32 rows, and their vote.
__device__ __forceinline__ void bar_pair(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
// the four warps of both tiles that hold the same 32 rows
__device__ __forceinline__ void bar_quad(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool bar_pair_or(int id, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)x), "r"(id)
                 : "memory");
    return r != 0;
}

// Item `item` of a sequence: tokens [tok0, tok1) of its rows, and the keys they see.
struct Item {
    int tok0, tok1, t0, nt;   // first key tile and number of tiles
    int lo, hi;
};
__host__ __device__ inline Item item_of(int item, int n, int kv, int window, int tokens) {
    Item x;
    x.tok0 = item * 2 * tokens;
    x.tok1 = x.tok0 + 2 * tokens < n ? x.tok0 + 2 * tokens : n;
    const int first = kv - n + x.tok0, last = kv - n + x.tok1 - 1;   // positions
    x.hi = last + 1 > 0 ? last + 1 : 0;
    x.lo = window > 0 && first - window + 1 > 0 ? first - window + 1 : 0;
    x.t0 = x.lo / kTile;
    x.nt = (x.hi + kTile - 1) / kTile - x.t0;
    if (x.nt < 1) x.nt = 1;
    return x;
}

// Unit `unit` of all items: a group of pairs after the other, within a group the
// last items of all its pairs first.  A causal prompt's last items are the longest,
// and long ones first lets the SMs end together (a 4K prompt of 32 heads: 134 us, pair
// by pair 147); a group has six waves of items or more, but few pairs, whose keys
// stay in L2 (a 16K prompt: 1349 us in two groups, 1430 in one).
__device__ __forceinline__ void unit_of(const TilePlan& plan, int unit, int pairs, int Hkv, int& b, int& h, int& item) {
    const int g0 = unit / (plan.group * plan.items) * plan.group, in = unit - g0 * plan.items;
    const int size = imin(plan.group, pairs - g0), back = in / size, pair = g0 + in - back * size;
    item = plan.items - 1 - back;
    b = pair / Hkv;
    h = pair - b * Hkv;
}

// NS: pages that half a tile of keys (64) touches, as far as scales go: 1, 2 or 4.
// One: no sequence has more rows than one tile.  The second tile then takes the
// same rows through every other tile of keys, and the two are joined at the end (16 rows of
// 4 heads, 32 sequences at 4K: 94 us, with the second tile idle 122; as a run-time choice
// it cost the chunks with two full tiles 2 to 5%).
template <bool E4, int D, int NS, bool One>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ PagedAttnParams p, const TilePlan plan) {
    using C = Cfg<E4, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sb = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kBars);
    const uint32_t abort_flag = sb + C::kOffBar + 8 * C::kBars + 4;
    auto bar_at = [&](int i) { return sb + C::kOffBar + 8u * (uint32_t)i; };
    const PagedView& c = p.c;
    const int G = p.G, tokens = kTile / G;   // tokens of a 128-row tile
    if (tid == 32) {
        tma_prefetch_map(&p.tm_q);
        tma_prefetch_map(&p.tm_k);
        tma_prefetch_map(&p.tm_v);
        st_shared_u32(abort_flag, 0u);
    }
    pdl_wait();
    pdl_trigger();
    // units [0, plan.whole) are whole items, the later ones are cut into splits
    const int over = (int)blockIdx.x - plan.whole;
    const int unit = over < 0 ? (int)blockIdx.x : plan.whole + over / plan.n_split, split = over < 0 ? 0 : over % plan.n_split;
    int b, h, item;
    unit_of(plan, unit, c.B * c.Hkv, c.Hkv, b, h, item);
    const SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, c.B, c.cap);
    const bool bad = !s.ok || s.n > p.max_rows || (sb & 1023u);
    if (bad && tid == 0 && p.status) atomicExch(p.status, MASW_EINVAL);
    const Item it = item_of(item, s.n, s.kv, p.window, tokens);
    const int n_split = over < 0 || it.nt < plan.min_tiles ? 1 : plan.n_split;
    const int chunk = (it.nt + n_split - 1) / n_split;
    const int j0 = split * chunk, nt = imin(it.nt, j0 + chunk) - j0;   // this CTA's tiles
    if (bad || item * 2 * tokens >= s.n || nt < 1) {                   // nothing to do (the merge knows of empty splits)
        return;
    }
    const int first_tile = it.t0 + j0;
    // the second tile has rows of its own
    const bool two = !One && it.tok1 - it.tok0 > tokens;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tslot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < C::kBars; ++i)
            mbar_init(bars + i, i >= C::kGo && i < C::kGo + 2                                                                ? 9
                                : (i >= C::kWFull && i < C::kWFree) || (E4 && i >= C::kVFree && i < C::kWFull)    ? 4
                                : two && ((i >= C::kKFree && i < C::kVFull) || (i >= C::kVFree && i < C::kMetaBar)) ? 2
                                                                                                                    : 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto wait = [&](int bar, int phase) { return wait_bounded(bar_at(bar), (uint32_t)phase & 1u, abort_flag, p.status); };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    bool ok = true;

    // 512 x 96 + 256 x 48 = 768 x 80 registers
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 16) {
            // ---------------- matrix products ----------------
            // one lane does it all: step k of tile x is P V of its tile of keys k - 1 and S
            // of its tile of keys k
            if (elect_one()) {
                uint32_t ks = 0, ws = 0;                 // stage of K, buffer of V
                auto step = [&](int x, int xq, int k, bool last, uint64_t bv, uint64_t bk) {
                    if (!wait(C::kGo + x, k)) return false;
                    tc_fence_after();
                    const uint64_t aq = E4 ? smem_desc(sb + C::kOffQ + xq * C::kTerms * C::kTileB, 128, (C::kRB / 16) * 128, 0)
                                           : smem_desc(sb + C::kOffQ + xq * C::kTileB, 16, 1024, 2);
                    const uint32_t ts = tmem + C::kColS + x * 128, to = tmem + C::kColO + x * 128;
                    if (k > 0) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            umma_bf16_ts(to, ts + (kk >> 2) * 64 + (kk & 3) * 8, bv + (uint64_t)((kk * 2048) >> 4), C::kIdescO, k > 1 || kk > 0);
                        umma_commit(bar_at((E4 ? C::kWFree : C::kVFree) + ws));
                        if (last) umma_commit(bar_at(C::kOFull + x));
                    }
                    if (!last) {
#pragma unroll
                        for (int t = 0; t < C::kTerms; ++t)
#pragma unroll
                            for (int kk = 0; kk < C::kRB / 32; ++kk) {
                                const uint32_t panel = (kk / (C::kPB / 32)) * C::kPanel + (kk % (C::kPB / 32)) * 32;
                                const uint64_t a = aq + (uint64_t)((E4 ? t * C::kTileB + kk * 256 : panel) >> 4);
                                const uint64_t bb = bk + (uint64_t)(panel >> 4);
                                if (E4) umma_f8(ts, a, bb, C::kIdescS, t > 0 || kk > 0);
                                else umma_bf16(ts, a, bb, C::kIdescS, t > 0 || kk > 0);
                            }
                        umma_commit(bar_at(C::kSFull + x));
                        umma_commit(bar_at(C::kKFree + ks));
                    }
                    return true;
                };
                auto v_at = [&]() { return smem_desc(sb + C::kOffW + ws * C::kWideB, C::kWPanel, 1024, 2); };
                auto k_at = [&]() { return smem_desc(sb + C::kOffK + ks * C::kTileB, 16, C::kAtom, C::kSwz); };
                if constexpr (One) {                     // key tiles 2 k + x - 2 and 2 k + x
                    for (int s = 0; ok && s < nt + 2; ++s) {
                        ok = step(s & 1, 0, s >> 1, s >= nt, v_at(), k_at());
                        ks = ks + 1 == C::kKS ? 0 : ks + 1;
                        if (s > 1) ws = ws + 1 == C::kWS ? 0 : ws + 1;
                    }
                } else {                                 // key tiles k - 1 and k
                    for (int k = 0; ok && k <= nt; ++k) {
                        const uint64_t bv = v_at(), bk = k_at();
                        for (int x = 0; ok && x < (two ? 2 : 1); ++x) ok = step(x, x, k, k == nt, bv, bk);
                        ks = ks + 1 == C::kKS ? 0 : ks + 1;
                        if (k > 0) ws = ws + 1 == C::kWS ? 0 : ws + 1;
                    }
                }
            }
            __syncwarp();
            ok = all(ok);
            // nothing may arrive on a barrier after the CTA ended
            if (ok) ok = all(wait(C::kKFree + (nt - 1) % C::kKS, (nt - 1) / C::kKS)) && all(wait((E4 ? C::kWFree : C::kVFree) + (nt - 1) % C::kWS, (nt - 1) / C::kWS));
            if (!ok) {
                st_shared_u32(abort_flag, 1u);
                if (elect_one()) umma_commit(bar_at(C::kDone));
                __syncwarp();
                mbar_wait(bars + C::kDone, 0, nullptr);
            }
        } else if (warp == 17) {
            // ---------------- K and V there: the ninth arrival on a step's barrier ----------------
            // (a test takes ~100 cycles: the issuing warp is left with one a step)
            if (elect_one()) {
                // Q: 128 / G tokens x G heads a tile (rows behind the sequence's are not
                // used, behind all rows they read as zeros)
                const int tiles = two ? 2 : 1;
                mbar_expect_tx_at(bar_at(C::kQLand), (uint32_t)(tiles * tokens * G * D * 2));
                for (int t = 0; t < tiles; ++t)
#pragma unroll
                    for (int pn = 0; pn < D / 64; ++pn)
                        tma_load_3d(sb + C::kOffLand + t * (C::kWPanels * C::kWPanel) + pn * C::kWPanel, &p.tm_q, pn * 64, h * G,
                                    s.r0 + it.tok0 + t * tokens, bar_at(C::kQLand));
            }
            __syncwarp();
            ok = all(wait(C::kQLand, 0));
            for (int s = 0; ok && s < nt + (One ? 2 : 1); ++s) {
                const int vt = s - (One ? 2 : 1);        // key tile of P V; that of S is s
                if (s < nt) ok = all(wait(C::kKFull + s % C::kKS, s / C::kKS));
                if (vt >= 0) ok = ok && all(wait(C::kWFull + vt % C::kWS, vt / C::kWS));
                for (int x = One ? s & 1 : 0; ok && x < (One ? (s & 1) + 1 : two ? 2 : 1); ++x) {
                    const int k = One ? s >> 1 : s;
                    if (k > 0) ok = all(wait(C::kGo + x, k - 1));   // one arrival a phase
                    if (ok && lane == 0) mbar_arrive(bar_at(C::kGo + x));
                }
            }
            if (!ok) {
                st_shared_u32(abort_flag, 1u);
                mbar_wait(bars + C::kQLand, 0, nullptr);   // no copy may be in flight when the CTA ends
            }
        } else if (warp < 20) {
            // ---------------- page ids, scales, TMA: warp 18 K, warp 19 V ----------------
            const bool is_v = warp == 19;
            const int stages = is_v ? C::kVS : C::kKS, full = is_v ? C::kVFull : C::kKFull, freed = is_v ? C::kVFree : C::kKFree;
            const uint32_t ring = sb + (is_v ? C::kOffV : C::kOffK);
            const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
            const bool scales = E4 && !is_v;
            const int box = imin(c.P, kTile), bpt = kTile / box, bt = 32 / bpt;
            const int key_lo = it.lo / c.P * c.P;    // first key of the first page with a visible key
            auto load_ids = [&](int j, int& pid, bool& in) {   // the boxes of tiles j .. j + bt - 1
                const int key = (first_tile + j) * kTile + lane * box;
                in = j < nt && lane < imin(bt, nt - j) * bpt && key < it.hi && key >= key_lo;
                pid = in ? __ldg(c.table + (size_t)b * c.table_stride + key / c.P) : 0;
            };
            auto check_and_scale = [&](int& pid, bool in, float& ks, float& vs) {
                if (in && (pid < 0 || pid >= c.n_pages)) {
                    if (p.status) atomicExch(p.status, MASW_EINVAL);
                    pid = 0;
                }
                ks = vs = 1.f;
                if (scales && in) {
                    ks = __ldg(c.k_scale + (size_t)pid * c.Hkv + h);
                    vs = __ldg(c.v_scale + (size_t)pid * c.Hkv + h);
                }
            };
            int pid, pid1, pid2, st = 0, turn = 0, issued = 0;
            bool in, in1, in2;
            float ks, vs, ks1, vs1;
            load_ids(0, pid, in);
            load_ids(bt, pid1, in1);
            check_and_scale(pid, in, ks, vs);
            for (int base = 0; ok && base < nt; base += bt) {
                check_and_scale(pid1, in1, ks1, vs1);
                load_ids(base + 2 * bt, pid2, in2);
                for (int j = base; j < imin(nt, base + bt); ++j) {
                    if (turn > 0) ok = all(wait(freed + st, turn - 1));
                    if (!ok) break;
                    const int q0 = (j - base) * bpt;
                    const uint32_t boxes = __ballot_sync(0xffffffffu, in) >> q0 & (bpt == 32 ? 0xffffffffu : (1u << bpt) - 1u);
                    if (elect_one()) mbar_expect_tx_at(bar_at(full + st), (uint32_t)(__popc(boxes) * box * C::kRB));
                    __syncwarp();
                    for (int q = 0; q < bpt; ++q) {
                        const int id = __shfl_sync(0xffffffffu, pid, q0 + q);
                        const int row = ((first_tile + j) * kTile + q * box) & (c.P - 1);
                        const uint32_t dst = ring + st * C::kTileB + (uint32_t)(q * box * C::kPB);
                        if ((boxes >> q & 1u) && elect_one()) {
#pragma unroll
                            for (int pn = 0; pn < C::kPanels; ++pn)
                                tma_load_4d(dst + pn * C::kPanel, map, pn * C::kPB / C::kES, row, h, id, bar_at(full + st));
                        }
                    }
                    __syncwarp();
                    if (scales) {   // behind the copies, which need not wait for them
                        if (lane >= q0 && lane < q0 + bpt)
                            st_shared_v4(sb + C::kOffMeta + (uint32_t)((j % kMeta) * 8 + lane - q0) * 16u, __float_as_uint(ks), __float_as_uint(vs == 1.f ? 0.f : __log2f(vs)), __float_as_uint(__frcp_rn(vs)), 0u);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_at(C::kMetaBar + j % kMeta));
                    }
                    ++issued;
                    if (++st == stages) {
                        st = 0;
                        ++turn;
                    }
                }
                pid = pid1;
                in = in1;
                ks = ks1;
                vs = vs1;
                pid1 = pid2;
                in1 = in2;
            }
            if (!ok) st_shared_u32(abort_flag, 1u);
            for (int k = imax(0, issued - stages); k < issued; ++k)
                mbar_wait(bars + full + k % stages, (uint32_t)(k / stages) & 1u, nullptr);
        } else {
            // ---------------- V as the products read it: thread t row t of the tile ----------------
            const int t = tid & 127;
            if (E4) ok = all(wait(C::kGo, 0)) && (!(One || two) || all(wait(C::kGo + 1, 0)));   // Q was read from where V goes
            for (int j = 0; ok && j < nt; ++j) {
                const int key = (first_tile + j) * kTile + t, st = j % C::kVS;
                const bool seen = key >= it.lo && key < it.hi;   // by some row; a row that none sees must not reach the product
                ok = all(wait(C::kVFull + st, j / C::kVS));
                if (E4 && j >= C::kWS) ok = ok && all(wait(C::kWFree + j % C::kWS, j / C::kWS - 1));
                if (!ok) break;
                const uint32_t dst = sb + C::kOffW + (j % C::kWS) * C::kWideB + t * 128;
                if constexpr (E4) {
                    const uint32_t src = sb + C::kOffV + st * C::kTileB + t * C::kPB;
                    const int swz = D == 128 ? t & 7 : (t >> 1) & 3;
#pragma unroll
                    for (int q0 = 0; q0 < D / 16; q0 += 4) {
                        float4 f[4];   // loads first: they are not reordered with the stores
#pragma unroll
                        for (int q = 0; q < 4; ++q) f[q] = ld_shared_v4f(src + ((uint32_t)((q0 + q) ^ swz) << 4));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[8];
                            e4m3x4_to_f16x2(__float_as_uint(f[q].x), w[0], w[1]);
                            e4m3x4_to_f16x2(__float_as_uint(f[q].y), w[2], w[3]);
                            e4m3x4_to_f16x2(__float_as_uint(f[q].z), w[4], w[5]);
                            e4m3x4_to_f16x2(__float_as_uint(f[q].w), w[6], w[7]);
                            if (!seen)
#pragma unroll
                                for (int e = 0; e < 8; ++e) w[e] = 0u;
                            const uint32_t at = dst + (uint32_t)((q0 + q) >> 2) * C::kWPanel;
                            st_shared_v4(at + (uint32_t)(((q * 2) ^ (t & 7)) << 4), w[0], w[1], w[2], w[3]);
                            st_shared_v4(at + (uint32_t)(((q * 2 + 1) ^ (t & 7)) << 4), w[4], w[5], w[6], w[7]);
                        }
                    }
                } else if (!seen) {
#pragma unroll
                    for (int pn = 0; pn < C::kWPanels; ++pn)
#pragma unroll
                        for (int q = 0; q < 8; ++q) st_shared_v4(dst + pn * C::kWPanel + q * 16, 0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_at(C::kWFull + j % C::kWS));
                    if (E4) mbar_arrive(bar_at(C::kVFree + st));
                }
            }
            if (!ok) st_shared_u32(abort_flag, 1u);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        // ---------------- softmax: row r of tile x, keys 64 hf .. 64 hf + 63 of each tile of keys ----------------
        const int x = warp >> 3, hf = (warp >> 2) & 1, r = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + C::kColS + x * 128 + lane_off, t_o = tmem + C::kColO + x * 128 + lane_off;
        const int pair = 1 + x * 4 + (warp & 3);                          // barrier of the two warps that share 32 rows
        float* slot = reinterpret_cast<float*>(smem + C::kOffRow) + x * kTile + r;
        // f of both halves' values, in both threads
        auto both = [&](float mine, auto f) {
            if (hf) *slot = mine;
            bar_pair(pair);
            if (!hf) *slot = mine = f(mine, *slot);
            bar_pair(pair);
            if (hf) mine = *slot;
            return mine;
        };
        const int tok_first = it.tok0 + (One ? 0 : x * tokens);           // of the tile
        const int tok_last = imin(it.tok1, tok_first + tokens) - 1;
        const int tok = imin(tok_first + r / G, tok_last), g = r % G;
        const int pos = s.kv - s.n + tok;
        const size_t row = (size_t)(s.r0 + tok) * p.Hq + (size_t)h * G + g;
        if (One || x == 0 || two) {
            // Q: this row's half, split into its terms
            float qs = 1.f;
            if constexpr (E4) {
                ok = wait(C::kQLand, 0);
                const int xq = One ? 0 : x;
                const uint32_t src = sb + C::kOffLand + xq * (C::kWPanels * C::kWPanel) + (D == 128 ? hf * C::kWPanel : 0) + r * 128;
                const uint32_t dst = sb + C::kOffQ + xq * C::kTerms * C::kTileB + (uint32_t)((r >> 3) * (C::kRB / 16) * 128 + (r & 7) * 16) +
                                     (uint32_t)(hf * (C::kRB / 32) * 128);
                auto chunk_of = [&](int k) {   // eight elements
                    const int ch = D == 128 ? k : hf * 4 + k;
                    return ld_shared_v4f(src + ((uint32_t)(ch ^ (r & 7)) << 4));
                };
                float amax = 0.f;
#pragma unroll 2
                for (int k = 0; k < D / 16; ++k) {
                    const float4 v = chunk_of(k);
                    float f[8];
                    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(&v), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(f[e]));
                }
                qs = pow2_scale(both(amax, [](float a, float b) { return fmaxf(a, b); }));
                const float inv = 1.f / qs;
                const int chunks = x == xq ? D / 16 : 0;   // the first tile's warps have split the rows of both
#pragma unroll 2
                for (int k = 0; k < chunks; ++k) {
                    const float4 v = chunk_of(k);
                    float f[8];
                    Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(&v), f);
                    uint32_t w1[2], w2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f0 = f[4 * e] * inv, f1 = f[4 * e + 1] * inv, f2 = f[4 * e + 2] * inv, f3 = f[4 * e + 3] * inv;
                        const uint32_t a = e4m3x2(f0, f1), bq = e4m3x2(f2, f3);
                        float d0, d1, d2, d3;
                        f16x2_to_f32(e4m3x2_to_f16x2(a), d0, d1);
                        f16x2_to_f32(e4m3x2_to_f16x2(bq), d2, d3);
                        w1[e] = a | (bq << 16);
                        w2[e] = e4m3x2(f0 - d0, f1 - d1) | (e4m3x2(f2 - d2, f3 - d3) << 16);
                    }
                    const uint32_t at = dst + (uint32_t)((k >> 1) * 128 + (k & 1) * 8);
                    st_shared_v2(at, w1[0], w1[1]);
                    st_shared_v2(at + C::kTileB, w2[0], w2[1]);
                }
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_at(C::kGo + x));
            const float qk = qs * p.scale_log2;
            const int row_lo = p.window > 0 ? imax(0, pos - p.window + 1) : 0;
            // keys that every row of the tile sees
            const int all_hi = s.kv - s.n + tok_first + 1;
            const int all_lo = p.window > 0 ? imax(0, s.kv - s.n + tok_last - p.window + 1) : 0;
            float mref = -INFINITY, l = 0.f;   // the row's reference (the same in both threads) and this half's sum
            constexpr int half = One ? 1 : 0;   // a tile takes every key tile, or every other one
            for (int j = half * x; j < nt; j += 1 + half) {
                const int tile0 = (first_tile + j) * kTile;
                float ks[NS], lvs[NS], ivs[NS];
                if constexpr (E4) {
                    ok &= wait(C::kMetaBar + j % kMeta, j / kMeta);
#pragma unroll
                    for (int q = 0; q < NS; ++q) {
                        const int box = NS > 1 ? hf * NS + q : (c.P >= kTile ? 0 : hf);
                        const float4 sc = ld_shared_v4f(sb + C::kOffMeta + (uint32_t)((j % kMeta) * 8 + box) * 16u);
                        ks[q] = qk * sc.x;
                        lvs[q] = sc.y;
                        ivs[q] = sc.z;
                    }
                } else {
                    ks[0] = qk;
                    lvs[0] = 0.f;
                }
                ok &= wait(C::kSFull + x, j >> half);
                __syncwarp();
                tc_fence_after();
                constexpr int kCols = kTile / 2;
                constexpr int kGroup = kCols / NS;   // columns of one page
                const bool masked = tile0 < all_lo || tile0 + kTile > all_hi;
                const int see_lo = row_lo - tile0 - hf * kCols, see_hi = pos + 1 - tile0 - hf * kCols;   // columns the row sees
                if (E4 && masked) {
                    // where the row sees nothing of a page, its scales may be anything
#pragma unroll
                    for (int q = 0; q < NS; ++q)
                        if (!((q + 1) * kGroup > see_lo && q * kGroup < see_hi)) {
                            ks[q] = ivs[q] = 1.f;
                            lvs[q] = 0.f;
                        }
                }
                // Weights relative to the row's reference, which moves when a score of
                // either half exceeds it by more than 2^kSlack: then they are computed
                // anew (rarely, so that nobody waits for the maximum to know).
                uint32_t w[kCols / 2];
                float sum;
#pragma unroll 1
                for (;;) {
                    float a[kCols];
                    tmem_ld_cols<kCols>(t_s + hf * 64, reinterpret_cast<uint32_t*>(a));
                    tmem_wait_ld();
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < kCols; ++e) a[e] = e >= see_lo && e < see_hi ? a[e] : -INFINITY;
                    }
                    const float nref = mref == -INFINITY ? 0.f : mref;
                    float mx = -INFINITY;
                    sum = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        const float add = lvs[n] - nref;
                        const uint64_t ks2 = f2_pack(ks[n], ks[n]), add2 = f2_pack(add, add);
                        uint64_t sum2 = 0, sum3 = 0;
                        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                        for (int e = n * kGroup; e < (n + 1) * kGroup; e += 4) {
                            m0 = fmax3(m0, a[e], a[e + 1]);
                            m1 = fmax3(m1, a[e + 2], a[e + 3]);
                            float u0, u1, u2, u3;
                            f2_unpack(f2_fma(f2_pack(a[e], a[e + 1]), ks2, add2), u0, u1);
                            f2_unpack(f2_fma(f2_pack(a[e + 2], a[e + 3]), ks2, add2), u2, u3);
                            u0 = ex2_approx(u0);
                            u1 = ex2_approx(u1);
                            u2 = ex2_approx(u2);
                            u3 = ex2_approx(u3);
                            sum2 = f2_add(sum2, f2_pack(u0, u1));
                            sum3 = f2_add(sum3, f2_pack(u2, u3));
                            w[e / 2] = E4 ? cvt_f16x2(u0, u1) : pack_bf16(u0, u1);
                            w[e / 2 + 1] = E4 ? cvt_f16x2(u2, u3) : pack_bf16(u2, u3);
                        }
                        float s0, s1;
                        f2_unpack(f2_add(sum2, sum3), s0, s1);
                        sum = E4 ? fmaf(s0 + s1, ivs[n], sum) : s0 + s1;
                        mx = fmaxf(mx, fmaf(fmaxf(m0, m1), ks[n], lvs[n]));
                    }
                    if (!bar_pair_or(pair, mx - mref > kSlack)) break;
                    const float top = both(mx, [](float a, float b) { return fmaxf(a, b); });
                    float alpha = 1.f;
                    if (top - mref > kSlack) {
                        const float up = top;
                        alpha = ex2_approx(mref - up);
                        mref = up;
                        l *= alpha;
                    }
                    if (j > half) {
                        // S(k) done means that P V of the tile before it is; this thread
                        // scales its half of the row's O
#pragma unroll 1
                        for (int q = hf * (D / 2); q < (hf + 1) * (D / 2); q += 16) {
                            uint32_t ov[16];
                            tmem_ld16(t_o + q, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            tmem_st16(t_o + q, ov);
                        }
                        tmem_wait_st();
                    }
                }
                l += sum;
                // P over the half of S that this thread read
                tmem_st16(t_s + hf * 64, *reinterpret_cast<uint32_t(*)[16]>(w));
                tmem_st16(t_s + hf * 64 + 16, *reinterpret_cast<uint32_t(*)[16]>(w + 16));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_at(C::kGo + x));
            }
            l = both(l, [](float a, float b) { return a + b; });
            float w0 = 1.f, w1 = 0.f;   // of this tile's outputs and, joined, of the second one's
            const bool join = One && nt > 1;
            if constexpr (One) {
                float* second = reinterpret_cast<float*>(smem + C::kOffRow) + kTile + r;
                if (x == 1 && hf == 0) {
                    second[0] = l;
                    second[kTile] = mref;
                }
                bar_quad(9 + (warp & 3));
                if (x == 0) {
                    const float l1 = second[0], m1 = second[kTile], m = fmaxf(mref, m1);
                    w0 = mref == -INFINITY ? 0.f : ex2_approx(mref - m);
                    w1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
                    l = l * w0 + l1 * w1;
                    mref = m;
                }
            }
            const bool mine = !One || x == 0;   // the outputs are this warp's to store
            const bool live = mine && r < (tok_last - tok_first + 1) * G;     // rows behind repeat the last token
            if (mine) ok &= wait(C::kOFull + x, 0);
            if (mine && join) ok &= wait(C::kOFull + 1, 0);
            __syncwarp();
            tc_fence_after();
            float* part = nullptr;
            if (n_split > 1) {
                part = p.part + (size_t)over * 256 * (D + 2) + x * 128 + r;   // [D + 2][256 rows]
                if (live && hf == 0) {
                    __stcg(part + D * 256, l == 0.f ? -INFINITY : mref);
                    __stcg(part + (D + 1) * 256, l);
                }
            } else if (live && hf == 0 && p.lse) {
                p.lse[row] = l == 0.f ? -INFINITY : (mref + __log2f(l)) * 0.6931471805599453f;
            }
            const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            w0 *= inv;
            w1 *= inv;
#pragma unroll 1
            for (int q = hf * (D / 2); q < (mine ? (hf + 1) * (D / 2) : 0); q += 32) {
                uint32_t ov[32];
                tmem_ld32(t_o + q, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * w0);
                if (join) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t o1[8];
                        tmem_ld8(t_o + 128 + q + e, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) ov[e + i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), w1, __uint_as_float(ov[e + i])));
                    }
                }
                if (!live) continue;
                if (part) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) __stcg(part + (q + e) * 256, __uint_as_float(ov[e]));
                } else if (p.o_f32) {
                    float* dst = reinterpret_cast<float*>(p.o) + row * D + q;
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        __stcg(reinterpret_cast<float2*>(dst + e), make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])));
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16(__uint_as_float(ov[8 * e + 2 * k]), __uint_as_float(ov[8 * e + 2 * k + 1]));
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
            if (!ok) st_shared_u32(abort_flag, 1u);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Joins the splits of an item: thread r row r of its 256, 8 elements a CTA, four
// splits' loads at a time (one sequence, 16 rows at 32K, 19 splits: 32 us; one by one, 32
// elements a CTA: 53).
constexpr int kMergeElems = 8, kAtOnce = 4;
template <int D>
__global__ void __launch_bounds__(256) tile_merge_kernel(const __grid_constant__ PagedAttnParams p, const TilePlan plan) {
    const PagedView& c = p.c;
    pdl_wait();
    pdl_trigger();
    const int G = p.G, tokens = kTile / G, n_split = plan.n_split, r = threadIdx.x;
    const int over = blockIdx.x, d0 = (int)blockIdx.y * kMergeElems;
    int b, h, item;
    unit_of(plan, plan.whole + over, c.B * c.Hkv, c.Hkv, b, h, item);
    const SeqRows s = seq_rows(p.row_start, p.kv_len, b, p.rows, c.B, c.cap);
    if (!s.ok || s.n > p.max_rows || item * 2 * tokens >= s.n) return;
    const Item it = item_of(item, s.n, s.kv, p.window, tokens);
    if (it.nt < plan.min_tiles) return;
    const int tok = it.tok0 + (r >> 7) * tokens + (r & 127) / G;
    if ((r & 127) >= tokens * G || tok >= it.tok1) return;
    const int chunk = (it.nt + n_split - 1) / n_split, pieces = (it.nt + chunk - 1) / chunk;
    float M = -INFINITY, l = 0.f, o[kMergeElems] = {};
    for (int q0 = 0; q0 < pieces; q0 += kAtOnce) {
        float m[kAtOnce], pl[kAtOnce], v[kAtOnce][kMergeElems];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int q = imin(q0 + k, pieces - 1);
            const float* part = p.part + ((size_t)over * n_split + q) * 256 * (D + 2) + r;
            m[k] = __ldcg(part + D * 256);
            pl[k] = __ldcg(part + (D + 1) * 256);
#pragma unroll
            for (int e = 0; e < kMergeElems; ++e) v[k][e] = __ldcg(part + (d0 + e) * 256);
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (q0 + k >= pieces) m[k] = -INFINITY;
            top = fmaxf(top, m[k]);
        }
        if (top == -INFINITY) continue;
        const float w = exp2f(M - top);
        l *= w;
#pragma unroll
        for (int e = 0; e < kMergeElems; ++e) o[e] *= w;
        M = top;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (m[k] == -INFINITY) continue;   // its outputs are not used, whatever they are
            const float wk = exp2f(m[k] - M);
            l = fmaf(pl[k], wk, l);
#pragma unroll
            for (int e = 0; e < kMergeElems; ++e) o[e] = fmaf(v[k][e], wk, o[e]);
        }
    }
    const size_t row = (size_t)(s.r0 + tok) * p.Hq + (size_t)h * G + (r & 127) % G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (p.o_f32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + row * D + d0);
        dst[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        dst[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + d0) =
            make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv), pack_bf16(o[4] * inv, o[5] * inv),
                       pack_bf16(o[6] * inv, o[7] * inv));
    }
    if (d0 == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.6931471805599453f;
}

template <bool E4, int D, int NS, bool One>
cudaError_t launch(const PagedAttnParams& p, const TilePlan& plan, cudaStream_t st) {
    using C = Cfg<E4, D>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(tile_kernel<E4, D, NS, One>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_release);
    }
    e = masw_launch(tile_kernel<E4, D, NS, One>, dim3(plan.whole + plan.cut * plan.n_split), dim3(kThreads), C::kSmem, st, 1, p, plan);
    if (e != cudaSuccess || plan.cut == 0) return e;
    return masw_launch(tile_merge_kernel<D>, dim3(plan.cut, D / kMergeElems), dim3(256), 0, st, 1, p, plan);
}

}  // namespace tile

cudaError_t launch_paged_tiles(const PagedAttnParams& p, const TilePlan& plan, cudaStream_t st) {
    auto pick = [&](auto e4, auto d, auto ns) {
        constexpr bool E4 = decltype(e4)::value;
        constexpr int D = decltype(d)::value, NS = decltype(ns)::value;
        return p.max_rows <= kTile / p.G ? tile::launch<E4, D, NS, true>(p, plan, st) : tile::launch<E4, D, NS, false>(p, plan, st);
    };
    auto by_dim = [&](auto e4, auto ns) {
        return p.c.D == 64 ? pick(e4, std::integral_constant<int, 64>{}, ns) : pick(e4, std::integral_constant<int, 128>{}, ns);
    };
    if (!p.c.k_scale) return by_dim(std::false_type{}, std::integral_constant<int, 1>{});
    if (p.c.P >= 64) return by_dim(std::true_type{}, std::integral_constant<int, 1>{});
    if (p.c.P == 32) return by_dim(std::true_type{}, std::integral_constant<int, 2>{});
    return by_dim(std::true_type{}, std::integral_constant<int, 4>{});
}

}  // namespace masw
