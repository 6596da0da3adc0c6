// Runs the step kernel's plan and walk (flint_paged_walk.cuh) on the host over
// random boundaries and lengths, and checks every index they make.  The arrays
// end at an inaccessible page, so a read past them ends the process.
//   paged_walk_host good|ill SEED CASES
#include <sys/mman.h>
#include <unistd.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../full_gqa_learned_b200/csrc/flint_paged_walk.cuh"

using namespace flint;

static const char* g_case = "";
static void check(bool ok, const char* what) {
    if (ok) return;
    std::printf("FAILED: %s\n%s\n", what, g_case);
    std::exit(1);
}

// n ints that end where an inaccessible page begins.
struct Guarded {
    int* at;
    char* base;
    size_t bytes;
    explicit Guarded(const std::vector<int>& v) {
        const size_t page = sysconf(_SC_PAGESIZE), need = v.size() * sizeof(int);
        bytes = (need + page - 1) / page * page;
        base = static_cast<char*>(mmap(nullptr, bytes + page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
        mprotect(base + bytes, page, PROT_NONE);
        bytes += page;
        at = reinterpret_cast<int*>(base + bytes - page - need);
        std::memcpy(at, v.data(), need);
    }
    ~Guarded() { munmap(base, bytes); }
};

struct Call {
    std::vector<int> cu, len;
    int T, max_new, max_pages, ps_log2, ng, window;
};

struct Pair { int b, row, head, tiles; };

template <int NT>
static void run(const Call& k, int tile) {
    const Guarded cu(k.cu), len(k.len);
    PagedAttnParams p = {};
    PagedCache& c = p.c;
    c.cu = cu.at;
    c.len = len.at;
    c.B = (int)k.len.size();
    c.T = k.T;
    c.max_pages = k.max_pages;
    c.num_pages = 1 << 20;
    c.ps_log2 = k.ps_log2;
    c.ng = k.ng;
    p.max_new = k.max_new;
    p.window = k.window;

    bool ill = c.cu[0] != 0;
    long long tiles = 0;
    for (int b = 0; b < c.B; ++b) tiles += step_seq_tiles<NT>(p, c.cu[b], c.cu[b + 1], c.len[b], tile, &ill);
    bool falls = c.cu[0] != 0 || c.cu[c.B] > c.T;
    for (int b = 0; b < c.B; ++b) falls = falls || c.cu[b + 1] < c.cu[b] || c.cu[b] < 0;
    check(!falls || ill, "ill-formed boundaries are reported");
    const long long W = tiles * c.ng, ctas = 296, G = W < ctas ? W : ctas;
    // the pairs in the order that the plan counts them
    std::vector<Pair> want;
    for (int b = 0; b < c.B; ++b) {
        const int n = paged_new(c, p.max_new, c.cu[b], c.cu[b + 1], c.len[b]);
        for (int r = 0; r < n; r += NT)
            for (int h = 0; h < c.ng; ++h) want.push_back({b, c.cu[b] + r, h, step_tiles(p, c.len[b] + r, min(NT, n - r), tile)});
    }
    size_t next = 0;
    int done = 0;                                            // tiles of want[next] that are taken
    for (long long cta = 0; cta < G; ++cta) {
        const long long t = W * cta / G, end = W * (cta + 1) / G;
        // the last CTA: also a share larger than what is left ends
        for (const int more : {0, 1000}) {
            if (more && cta + 1 < G) continue;
            int at[4] = {-1, -1, -1, -1};
            step_place<NT>(p, 0, c.B, t, tile, at);
            check(at[0] >= 0 && at[0] < c.B, "the share begins at a sequence");
            StepWalk w = {};
            step_begin(p, w, at, (int)(end - t) + more, ill);
            StepSeg s;
            long long taken = 0, steps = 0;
            while (step_next<NT>(p, w, s, tile)) {
                check(++steps <= end - t + (more ? (long long)want.size() : 0), "a share has at most as many pairs as tiles");
                check(s.b >= 0 && s.b < c.B && s.head >= 0 && s.head < c.ng, "sequence and head");
                check(s.nrows >= 1 && s.nrows <= NT && s.row >= 0 && s.row + s.nrows <= c.T, "rows");
                check(s.p0 >= 0 && (long long)s.p0 + s.nrows <= FLINT_MAX_TOKENS &&
                          ((s.p0 + s.nrows - 1) >> c.ps_log2) < c.max_pages, "positions within the page table");
                check(s.t0 >= 0 && s.t0 < s.t1 && s.t1 <= s.tiles, "tiles of the pair");
                if (more) continue;
                taken += s.t1 - s.t0;
                check(next < want.size(), "a pair that the plan counted");
                const Pair& q = want[next];
                check(q.b == s.b && q.row == s.row && q.head == s.head && q.tiles == s.tiles && done == s.t0, "the pair that is next");
                done = s.t1;
                if (done == s.tiles) {
                    ++next;
                    done = 0;
                }
            }
            check(more || taken == end - t, "the whole share is walked");
        }
    }
    check(next == want.size() && done == 0, "every pair is walked");
}

static std::string text(const Call& k) {
    std::string s = "cu";
    for (int x : k.cu) s += " " + std::to_string(x);
    s += "; len";
    for (int x : k.len) s += " " + std::to_string(x);
    return s + "; T " + std::to_string(k.T) + " max_new " + std::to_string(k.max_new) + " max_pages " + std::to_string(k.max_pages) +
           " page " + std::to_string(1 << k.ps_log2) + " heads " + std::to_string(k.ng) + " window " + std::to_string(k.window);
}
static void both(const Call& k) {
    const std::string s = text(k);
    g_case = s.c_str();
    run<2>(k, 64);
    run<2>(k, 128);
    Call one = k;
    one.max_new = k.max_new < 1 ? k.max_new : 1;
    run<1>(one, 64);
    run<1>(one, 128);
    g_case = "";
}

int main(int argc, char** argv) {
    if (argc != 4) return 2;
    const bool bad = !std::strcmp(argv[1], "ill");
    std::mt19937 rng(std::atoi(argv[2]));
    auto pick = [&](int lo, int hi) { return (int)(rng() % (unsigned)(hi - lo + 1)) + lo; };
    if (bad) {
        both({{0, 2, 2, 2, 4, 2, 2}, {100000, 0, 0, 50000, 0, 0}, 4, 2, 2000, 6, 4, 0});
        both({{0, 2, 2, 2, 4, 2, 2}, {100000, 0, 0, 50000, 0, 5000000}, 4, 2, 2000, 6, 4, 0});
        both({{0, 2, 7, 0, 4, 2}, {9000, 100, 100, 20000, 0}, 8, 4, 2000, 4, 1, 0});
    }
    for (int i = std::atoi(argv[3]); i > 0; --i) {
        Call k;
        const int B = pick(0, 9) ? pick(1, 12) : pick(30, 400);
        k.max_new = pick(0, 8);
        k.ps_log2 = pick(4, 7);
        k.ng = 1 << pick(0, 2);
        k.window = pick(0, 1) ? 0 : pick(1, 700);
        k.max_pages = pick(1, 60);
        const int idle = pick(0, 3);
        k.cu.push_back(0);
        for (int b = 0; b < B; ++b) {
            const int n = pick(0, 3) < idle ? 0 : pick(0, k.max_new);
            const int room = max(0, (k.max_pages << k.ps_log2) - n);
            k.len.push_back(pick(0, 3) ? pick(0, room) : min(room, pick(0, 40)));
            k.cu.push_back(k.cu.back() + n);
        }
        k.T = k.cu.back() + pick(0, 3);
        if (bad) {
            for (int j = pick(1, 4); j > 0; --j) {
                const int b = pick(0, B), what = pick(0, 5);
                if (what == 0) k.cu[b] = pick(0, k.T);
                else if (what == 1) k.cu[b] = pick(0, 1) ? -pick(1, 5) : k.T + pick(0, 900);
                else if (what == 2) for (int x = b; x <= min(B, b + pick(1, 6)); ++x) k.cu[x] = k.cu[b] + pick(-1, 1) * pick(0, 2);
                else if (what == 3) k.len[min(b, B - 1)] = pick(0, 1) ? -pick(1, 1 << 30) : pick(0, 0x7fffffff);
                else if (what == 4) for (int x = 0; x <= B; x += pick(1, 3)) k.cu[x] = pick(0, k.T);
                else k.cu[b] = pick(0, 1) ? 0x7fffffff : -0x7fffffff - 1;
            }
        }
        both(k);
    }
    std::printf("OK\n");
    return 0;
}
