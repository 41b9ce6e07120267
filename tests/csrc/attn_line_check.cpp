// Host checks of the cut of attention's line of tiles, built from the plan
// kernel's own header (moe_expert_cache_gb300/csrc/attn_line.cuh).  Over
// random lines and over the longest ones that the entry points accept
// (prompts whose cost passes 2^31, with few and many query heads a key/value
// head, and segments of 2^24 tiles):
//   * the parts of the CTAs are ascending and cover the whole line;
//   * every tile of every segment is in one CTA, a segment's tiles lie in
//     consecutive CTAs, and the first of them are in the CTA that holders()
//     names first, the last in the one that it names last;
//   * a CTA continues at most one segment of another (its partial result has
//     one place per CTA), its items are as many as items() says, and all items
//     together are no more than a segment's one each and one more per CTA;
//   * no CTA has more of the line than its even share and a rest.
// Exits 0 and prints "ok", or prints the first failure and exits 1.
#include "attn_line.cuh"

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

using namespace attnline;

namespace {

[[noreturn]] void fail(const char* what, long long a, long long b) {
    std::printf("FAIL %s %lld %lld\n", what, a, b);
    std::exit(1);
}

unsigned rnd(unsigned& s) {
    s = s * 1664525u + 1013904223u;
    return s >> 8;
}

void check(const std::vector<int>& ntile, int Hkv, int n_cta, int n_items, int c) {
    const int n_seg = (int)ntile.size();
    std::vector<cost_t> cum(n_seg);
    cost_t cost = 0;
    __int128 exact = 0;
    for (int i = 0; i < n_seg; ++i) {
        cum[i] = cost;
        cost += segment_cost(ntile[i]);
        exact += (__int128)ntile[i] + OV;
        if ((__int128)cost != exact) fail("cost", i, (long long)cost);
    }
    auto cum_of = [&](int i) { return cum[i]; };
    const Line line(cost, Hkv, n_seg, n_cta, n_items, c);
    if ((__int128)line.S != exact * Hkv || line.start_of(0) != 0 || line.start_of(n_cta) != line.S)
        fail("ends", line.S, line.start_of(n_cta));
    long long n_works = 0;
    int next = 0, done = 0;       // segment of all heads and how many of its tiles are taken
    int held0 = -1, held1 = -1;   // CTAs that took the current segment's first and last tiles
    const long long n_all = (long long)n_seg * Hkv;
    for (int i = 0; i < n_cta; ++i) {
        const long long x0 = line.start_of(i), x1 = line.start_of(i + 1);
        if (x1 < x0) fail("descending part", i, x1 - x0);
        const long long share = i < line.n1 ? line.q1 : line.q0;
        if (x1 - x0 > share) fail("share", x1 - x0, share);
        if (x1 == x0) continue;
        const int l0 = line.at(x0, cum_of), l1 = line.at(x1 - 1, cum_of);
        if (l0 < 0 || l1 < l0 || l1 >= n_all) fail("range", l0, l1);
        const int want = Line::items(l0, l1, line.begin_of(l1, cum_of), x1);
        int got = 0, continued = 0;
        for (int l = l0; l <= l1; ++l) {
            const int nt = ntile[l % n_seg];
            int t0, t1;
            Line::tiles(line.begin_of(l, cum_of), nt, x0, x1, t0, t1);
            if (t0 >= t1) {
                if (l != l1) fail("empty item before the last", i, l);
                continue;
            }
            ++got;
            if (l != next || t0 != done || t1 > nt) fail("tiles", l, t0);
            if (t0 == 0) held0 = i;
            if (t0 > 0) ++continued;
            done = t1;
            if (done == nt) {
                held1 = i;
                int c0, c1;
                line.holders(line.begin_of(l, cum_of), nt, c0, c1);
                if (c0 != held0 || c1 != held1) fail("holders", c0 - held0, c1 - held1);
                ++next;
                done = 0;
            }
        }
        if (got != want) fail("items", got, want);
        if (continued > 1) fail("continued", i, continued);
        n_works += got;
    }
    if (next != n_all || done != 0) fail("covered", next, done);
    if (n_works > n_all + n_cta) fail("works", n_works, n_all);
}

// A causal prompt of T tokens behind `before` ones: segments of 128 rows, G rows a token.
std::vector<int> prompt(long long T, int G, long long before) {
    std::vector<int> nt;
    for (long long r0 = 0; r0 < T * G; r0 += 128) {
        const long long r1 = r0 + 127 < T * G - 1 ? r0 + 127 : T * G - 1;
        nt.push_back((int)((before + r1 / G + 1 + 127) / 128));
    }
    return nt;
}

}  // namespace

int main() {
    unsigned s = 1;
    for (int it = 0; it < 3000; ++it) {
        std::vector<int> nt(1 + rnd(s) % 60);
        const unsigned most = 1u << rnd(s) % 12;
        for (int& x : nt) x = 1 + rnd(s) % most;
        const int Hkv = 1 + rnd(s) % 5, n_cta = 1 + rnd(s) % 40;
        const int n_items = rnd(s) % 2 ? rnd(s) % (4 * n_cta) : 0;
        check(nt, Hkv, n_cta, n_items, 1 + rnd(s) % 50);
    }
    for (int n_cta : {152, 304}) {
        check(prompt(12000, 8, 8192), 4, n_cta, 0, 1);
        check(prompt(741000, 128, 0), 1, n_cta, 0, 1);
        check(prompt(1100000, 64, 0), 1, n_cta, 0, 1);
        check(prompt(2100000, 16, 0), 2, n_cta, 0, 1);
        check(prompt(3000000, 8, 0), 8, n_cta, 0, 1);
        check(prompt(20000, 128, (1ll << 31) - 30000), 4, n_cta, 77, 3);
        check(std::vector<int>(1024, 1 << 24), 64, n_cta, 4 * n_cta, 1000);
    }
    std::printf("ok\n");
    return 0;
}
