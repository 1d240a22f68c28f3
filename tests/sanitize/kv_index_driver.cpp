// kv_index_driver.cpp -- the attention kernels' integer work on the host: for
// random calls, well-formed and not, every key that a query sees is computed
// by exactly one chunk, every row that would be read lies inside the cache's
// bytes, no table entry outside the table is looked at, and every partial
// result lies inside the planned workspace.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "fp4q_attend_index.h"

using namespace fp4q;

static std::mt19937 rng(7);
static int pick(int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); }
#define CHECK(x) do { if (!(x)) { std::printf("case %d: failed: %s (line %d)\n", turn, #x, __LINE__); return 1; } } while (0)

int main()
{
    for (int turn = 0; turn < 3000; ++turn) {
        AttendArgs a{};
        const bool odd = turn % 3 == 2; // some lengths, starts and pages are wrong
        a.kv.mx = pick(0, 1);
        a.kv.head_dim = 64 << pick(0, 2);
        a.kv.heads = pick(1, 4);
        const bool paged = pick(0, 1);
        a.kv.page_size = paged ? 16 * pick(1, 5) : pick(1, 700);
        a.batch = pick(1, 6);
        a.group = pick(1, 20);
        a.q_heads = a.group * a.kv.heads;
        a.causal = pick(0, 3) != 0;
        a.window = a.causal && pick(0, 1) ? pick(1, 300) : 0;
        a.max_kv = paged ? pick(0, 900) : pick(0, a.kv.page_size);
        a.max_q = pick(1, 40);
        a.bf16 = pick(0, 1);
        const int tokens = a.kv.page_size, dim = a.kv.head_dim, block = a.kv.mx ? 32 : 16;
        a.kv.num_pages = paged ? pick(1, 60) : a.batch - (odd ? pick(0, 1) : 0);
        // heads inside tokens or tokens inside heads
        const bool nhd = pick(0, 1);
        const int64_t crow = dim / 2, srow = dim / block;
        a.kv.c_token = nhd ? crow * a.kv.heads : crow;
        a.kv.c_head = nhd ? crow : crow * tokens;
        a.kv.c_page = crow * tokens * a.kv.heads;
        a.kv.s_token = nhd ? srow * a.kv.heads : srow;
        a.kv.s_head = nhd ? srow : srow * tokens;
        a.kv.s_page = srow * tokens * a.kv.heads;
        const int64_t cbytes = a.kv.c_page * a.kv.num_pages, sbytes = a.kv.s_page * a.kv.num_pages;

        std::vector<int32_t> lens, starts{0}, table;
        for (int b = 0; b < a.batch; ++b) {
            lens.push_back(odd && pick(0, 2) == 0 ? pick(-5, 3000) : pick(0, a.max_kv));
            starts.push_back(starts.back() + pick(0, a.max_q + (odd ? 5 : 0)));
        }
        a.total_q = starts.back();
        if (odd && pick(0, 1))
            starts[pick(0, a.batch)] += pick(-9, 9);
        a.table_len = paged ? (a.max_kv + tokens - 1) / tokens + pick(0, 2) : 0;
        a.table_stride = a.table_len;
        table.resize((size_t)a.batch * a.table_len);
        for (int32_t& t : table)
            t = odd && pick(0, 9) == 0 ? pick(-3, 200) : pick(0, (int)a.kv.num_pages - 1);
        a.table = paged ? table.data() : nullptr; // sanitizers watch its ends
        a.kv_lens = lens.data();
        a.q_starts = starts.data();

        const AttendPlan p = plan_of(a);
        CHECK(p.chunks >= 1 && p.chunk % kStepKeys == 0 && (p.many || p.chunk <= kMaxChunk));
        CHECK((int64_t)p.tiles * p.rows_per_tile >= (int64_t)a.max_q * a.group);
        const int64_t all = (int64_t)a.batch * a.kv.heads * a.max_q * a.group * p.chunks;
        if (p.chunks > 1)
            CHECK(p.workspace >= (size_t)(((all * 8 + 255) & ~(int64_t)255) + all * dim * 4));
        for (int b = 0; b < a.batch; ++b) {
            const Extent e = extent_of(a, b);
            const int rows = e.qn * a.group;
            CHECK(e.qn >= 0 && e.qn <= a.max_q);
            CHECK(e.qn == 0 || (e.q0 >= 0 && e.q0 + e.qn <= a.total_q));
            const int head = pick(0, a.kv.heads - 1);
            for (int tile = 0; tile < p.tiles; ++tile) {
                const int r0 = tile * p.rows_per_tile;
                if (r0 >= rows)
                    continue;
                const int r1 = std::min(rows, r0 + p.rows_per_tile);
                int lo, hi;
                tile_keys(a, e, r0, r1, lo, hi);
                const int chunks = chunks_of(p, lo, hi);
                CHECK(chunks <= p.chunks);
                std::vector<int> count(e.kn + 64, 0);
                for (int c = 0; c < chunks; ++c) {
                    const int k0 = lo + c * p.chunk;
                    const int k1 = hi - k0 < p.chunk ? hi : k0 + p.chunk;
                    CHECK(k0 % 32 == 0 && (p.many || k1 - k0 <= kMaxChunk));
                    for (int key = k0; key < k1; key += 16) {
                        const Granule g = granule_at(a, b, head, key);
                        const int n = std::min(16, k1 - key);
                        for (int i = 0; i < n; ++i)
                            ++count[key + i];
                        CHECK((g.codes < 0) == (g.scales < 0));
                        if (g.codes < 0) {
                            CHECK(odd);
                            continue;
                        }
                        CHECK(g.codes % 16 == 0);
                        CHECK(g.codes + (n - 1) * a.kv.c_token + crow <= cbytes);
                        CHECK(g.scales + (n - 1) * a.kv.s_token + srow <= sbytes);
                    }
                }
                for (int r = r0; r < r1; ++r) {
                    int s0, s1;
                    seen_by(a, e, r / a.group, s0, s1);
                    CHECK(s0 >= 0 && s1 <= e.kn);
                    const int n = starts[b + 1] - starts[b];
                    const int last = a.causal ? std::max(0, e.kn - n + r / a.group + 1) : e.kn;
                    CHECK(s1 == last && s0 == (a.window ? std::max(0, last - a.window) : 0));
                    for (int k = s0; k < s1; ++k)
                        CHECK(count[k] == 1);
                }
            }
        }
    }
    std::printf("3000 calls indexed clean\n");
    return 0;
}
