// Host checks of the paged-cache calls' index arithmetic, built and run by
// test_paged_host.py; prints one "name value" line per check.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <set>
#include <vector>

#include "../compressed_draft_kv_gb300/csrc/masw_paged.cuh"

using namespace masw;

int main() {
    std::mt19937 g(7);
    auto upto = [&](int n) { return (int)(g() % (unsigned)(n + 1)); };
    // every (sequence, touched page) has exactly one unit, inside the grid
    long batches = 0, lost = 0, outside = 0, twice = 0;
    for (int rep = 0; rep < 600; ++rep, ++batches) {
        const int P = 16 << upto(4), B = 1 + upto(20), first = upto(30);
        std::vector<int> rs(1, first), kv;
        for (int b = 0; b < B; ++b) {
            const int n = upto(3) == 0 ? 0 : upto(rep % 2 ? 5 : 300);
            rs.push_back(rs.back() + n);
            kv.push_back(n + upto(500));
        }
        const int rows = rs.back() + upto(9), units = append_units(rows, B, P);
        std::set<std::pair<int, int>> seen;
        for (int u = 0; u < units; ++u) {
            int b = 0;
            for (int i = 0; i < B; ++i)
                if (append_unit_base(rs[i], i, P) <= u) b = i;
            const SeqRows s = seq_rows_of(rs[b], rs[b + 1], kv[b], rows, 1 << 20);
            if (s.n < 1) continue;
            const int lp = u - append_unit_base(s.r0, b, P), page = (s.kv - s.n) / P + lp;
            if (lp < 0 || page > (s.kv - 1) / P) continue;
            if (!seen.insert({b, page}).second) ++twice;
        }
        for (int b = 0; b < B; ++b)
            for (int p = kv[b] - (rs[b + 1] - rs[b]); p < kv[b]; ++p)
                if (!seen.count({b, p / P})) ++lost;
        for (const auto& x : seen)
            if (x.second > (kv[x.first] - 1) / P) ++outside;
    }
    std::printf("batches %ld\nlost %ld\noutside %ld\ntwice %ld\n", batches, lost, outside, twice);
    // bad ranges and lengths are told apart and carry no rows
    int accepted = 0;
    const int bad[][5] = {{-1, 2, 5, 9, 64}, {3, 2, 5, 9, 64}, {3, 10, 12, 9, 64}, {0, 1, -1, 9, 64}, {0, 1, 65, 9, 64}};
    for (const auto& x : bad) {
        const SeqRows s = seq_rows_of(x[0], x[1], x[2], x[3], x[4]);
        accepted += s.ok || s.n != 0 || s.kv != 0;
    }
    std::printf("bad_ranges_accepted %d\n", accepted);
    // scale exponents against a search
    long scales = 0, wrong = 0;
    for (int i = 0; i < 4000; ++i, ++scales) {
        float a = std::ldexp((float)(1 + upto(1 << 24)) / (1 << 24), upto(250) - 150);
        if (i % 4 == 0) a = std::ldexp(1.75f, upto(200) - 100);
        if (i % 4 == 1) a = std::nextafterf(std::ldexp(1.75f, upto(200) - 100), 1e38f);
        if (a == 0.f) continue;
        uint32_t bits;
        std::memcpy(&bits, &a, 4);
        int e = -64;
        while (e < 119 && (double)a > 448.0 * std::ldexp(1.0, e)) ++e;
        wrong += pow2_scale_exp(bits) != e;
    }
    // shares of tiles: every tile once, its owner found again
    long torn = 0;
    for (int i = 0; i < 3000; ++i) {
        const int C = 1 + upto(200), total = upto(i % 2 ? 300 : 200000), nt = 1 + upto(i % 2 ? 20 : 5000), s = 1 + upto(160);
        torn += first_tile(0, total, C) != 0 || first_tile(C, total, C) != total;
        for (int c = 0; c < C; ++c) {
            const int a = first_tile(c, total, C), b = first_tile(c + 1, total, C);
            torn += b < a || b - a > total / C + 1;
            if (b > a) torn += tile_owner(a, total, C) != c || tile_owner(b - 1, total, C) != c;
        }
        torn += part_first(0, nt, s) != 0 || part_first(s, nt, s) != nt;
        for (int k = 0; k < s; ++k) {
            const int n = part_first(k + 1, nt, s) - part_first(k, nt, s);
            torn += n < 0 || n > (nt + s - 1) / s || (n > 0) != (k < nt);
        }
        const int pairs = 1 + upto(300), own = pair_ctas(pairs, nt, total, C);
        torn += own < 0 || own * pairs > C || (own && (nt + own - 1) / own > total / C + kUneven);
    }
    std::printf("torn_shares %ld\n", torn);
    std::printf("scales %ld\nwrong_scales %ld\nzero_scale %d\n", scales, wrong, pow2_scale_exp(0));
    return 0;
}
