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
        a.kv.page_size = paged ? 16 * pick(1, 5) : pick(1, 1700);
        a.batch = pick(1, 6);
        a.group = pick(1, 20);
        a.q_heads = a.group * a.kv.heads;
        a.causal = pick(0, 3) != 0;
        a.window = a.causal && pick(0, 1) ? pick(1, 300) : 0;
        a.max_kv = paged ? pick(0, 2900) : pick(0, a.kv.page_size);
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
            lens.push_back(odd && pick(0, 2) == 0 ? pick(-5, 6000) : pick(0, a.max_kv));
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

        a.rotate = pick(0, 1) ? block : 0;
        const AttendPlan p = plan_of(a);
        CHECK(p.groups > 0 && p.chunks >= 1);
        CHECK((int64_t)p.tiles * p.rows_per_tile >= (int64_t)a.max_q * a.group);
        const int64_t pairs = (int64_t)a.batch * a.kv.heads;
        // keys computed, by sequence and KV head and row tile
        std::vector<std::vector<int>> count((size_t)pairs * p.tiles, std::vector<int>(a.max_kv + 64, 0));
        auto compute = [&](int b, int head, int tile, int k0, int k1) {
            if (k0 % 32 != 0)
                return false;
            for (int key = k0; key < k1; key += 16) {
                const Granule g = granule_at(a, b, head, key);
                const int n = std::min(16, k1 - key);
                for (int i = 0; i < n; ++i)
                    ++count[((size_t)b * a.kv.heads + head) * p.tiles + tile][key + i];
                if ((g.codes < 0) != (g.scales < 0))
                    return false;
                if (g.codes < 0) {
                    if (!odd)
                        return false;
                    continue;
                }
                if (g.codes % 16 != 0 || g.codes + (n - 1) * a.kv.c_token + crow > cbytes ||
                    g.scales + (n - 1) * a.kv.s_token + srow > sbytes)
                    return false;
            }
            return true;
        };
        int64_t places = 0;
        if (p.many) {
            CHECK(p.chunk % 64 == 0);
            for (int b = 0; b < a.batch; ++b) {
                const Extent e = extent_of(a, b);
                const int rows = e.qn * a.group;
                for (int tile = 0; tile < p.tiles; ++tile) {
                    const int r0 = tile * p.rows_per_tile;
                    if (r0 >= rows)
                        continue;
                    int lo, hi;
                    tile_keys(a, e, r0, std::min(rows, r0 + p.rows_per_tile), lo, hi);
                    CHECK(chunks_of(p, lo, hi) <= p.chunks);
                    for (int head = 0; head < a.kv.heads; ++head)
                        for (int c = 0; c < chunks_of(p, lo, hi); ++c) {
                            const int k0 = lo + c * p.chunk;
                            CHECK(compute(b, head, tile, k0, hi - k0 < p.chunk ? hi : k0 + p.chunk));
                        }
                }
            }
            places = pairs * a.max_q * a.group * p.chunks;
        } else {
            // the workgroups' parts, and each pair's partial results as the joining kernel finds them
            uint32_t total = 0;
            for (int b = 0; b < a.batch; ++b)
                total += (uint32_t)few_steps(a, extent_of(a, b)) * a.kv.heads;
            CHECK(p.groups == pairs + p.parts && (p.chunks == 1) == (p.parts == 0));
            const uint32_t most = p.chunks == 1 ? 0 : few_most(p, total) + pick(0, 20); // the kernel may lengthen parts
            int64_t parts_all = 0, slots_all = 0;
            for (int b = 0; b < a.batch; ++b) {
                const Extent e = extent_of(a, b);
                const uint32_t steps = few_steps(a, e);
                CHECK((steps == 0) == (e.qn == 0));
                if (steps == 0)
                    continue;
                int lo = 0, hi = 0;
                tile_keys(a, e, 0, e.qn * a.group, lo, hi);
                for (int head = 0; head < a.kv.heads; ++head) {
                    if (p.chunks == 1) {
                        CHECK(compute(b, head, 0, lo, hi));
                        continue;
                    }
                    const uint32_t parts = few_parts(steps, most);
                    parts_all += parts;
                    slots_all += parts > 1 ? parts : 0;
                    for (uint32_t i = 0; i < parts; ++i) {
                        const int from = few_from(steps, parts, i), to = few_from(steps, parts, i + 1);
                        CHECK(from < to && to - from <= (int)most && (i > 0 || from == 0));
                        CHECK(compute(b, head, 0, lo + from * kStepKeys, to == (int)steps ? hi : lo + to * kStepKeys));
                    }
                }
            }
            CHECK(p.chunks == 1 || (parts_all <= p.groups && slots_all <= 2 * p.parts));
            places = (int64_t)2 * p.parts * p.rows_per_tile;
        }
        if (p.chunks > 1)
            CHECK(p.workspace >= (p.many ? 0 : few_table_bytes(p.groups, a.batch) + round256((size_t)pairs * 8)) + round256((size_t)places * 8) + (size_t)places * dim * 4);
        for (int b = 0; b < a.batch; ++b) {
            const Extent e = extent_of(a, b);
            CHECK(e.qn >= 0 && e.qn <= a.max_q);
            CHECK(e.qn == 0 || (e.q0 >= 0 && e.q0 + e.qn <= a.total_q));
            for (int r = 0; r < e.qn * a.group; ++r) {
                int s0, s1;
                seen_by(a, e, r / a.group, s0, s1);
                CHECK(s0 >= 0 && s1 <= e.kn);
                const int n = starts[b + 1] - starts[b];
                const int last = a.causal ? std::max(0, e.kn - n + r / a.group + 1) : e.kn;
                CHECK(s1 == last && s0 == (a.window ? std::max(0, last - a.window) : 0));
                for (int head = 0; head < a.kv.heads; ++head)
                    for (int k = s0; k < s1; ++k)
                        CHECK(count[((size_t)b * a.kv.heads + head) * p.tiles + r / p.rows_per_tile][k] == 1);
            }
        }
    }
    std::printf("3000 calls indexed clean\n");
    return 0;
}
