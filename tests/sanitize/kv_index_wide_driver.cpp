// kv_index_wide_driver.cpp -- the attention kernels' integer work at sizes past
// kv_index_driver.cpp's: hundreds of sequences, whose parts are written down in
// the workspace first, contexts of many chunks, and the rows before a window.
// The table is laid out in a buffer of exactly the planned bytes, which the
// sanitizers watch.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "fp4q_attend_index.h"

using namespace fp4q;

static std::mt19937 rng(11);
static int pick(int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); }
#define CHECK(x) do { if (!(x)) { std::printf("case %d: failed: %s (line %d)\n", turn, #x, __LINE__); return 1; } } while (0)

int main()
{
    int tables = 0, most_chunks = 0, windows = 0;
    for (int turn = 0; turn < 1500; ++turn) {
        AttendArgs a{};
        const bool odd = turn % 3 == 2;
        const bool crowd = turn % 2 == 0; // many sequences, few queries
        a.kv.mx = pick(0, 1);
        a.kv.head_dim = 64 << pick(0, 2);
        a.kv.heads = pick(1, crowd ? 4 : 2);
        a.kv.page_size = 16 * pick(1, 5);
        a.kv.num_pages = 1 << 30; // places are not looked up here
        a.batch = crowd ? pick(200, 900) : pick(1, 3);
        a.group = pick(1, crowd ? 8 : 20);
        a.q_heads = a.group * a.kv.heads;
        a.causal = pick(0, 3) != 0;
        a.window = a.causal && pick(0, 1) ? pick(1, 5000) : 0;
        a.max_kv = pick(0, crowd ? 9000 : 200000);
        a.max_q = crowd ? pick(1, 64 / a.group) : pick(1, 400);
        a.bf16 = pick(0, 1);
        a.rotate = pick(0, 1) ? (a.kv.mx ? 32 : 16) : 0;
        std::vector<int32_t> lens, starts{0};
        for (int b = 0; b < a.batch; ++b) {
            const int some = crowd && pick(0, 9) ? std::min(a.max_kv, 300) : a.max_kv;
            lens.push_back(odd && pick(0, 9) == 0 ? pick(-5, 1 << 30) : pick(0, some));
            starts.push_back(starts.back() + pick(0, a.max_q + (odd ? 5 : 0)));
        }
        a.total_q = starts.back();
        if (odd)
            starts[pick(0, a.batch)] += pick(-9, 9);
        a.table_len = (a.max_kv + a.kv.page_size - 1) / a.kv.page_size;
        a.table_stride = a.table_len;
        std::vector<int32_t> table(1);
        a.table = table.data();
        a.kv_lens = lens.data();
        a.q_starts = starts.data();
        const AttendPlan p = plan_of(a);
        CHECK(p.groups > 0);
        const int64_t pairs = (int64_t)a.batch * a.kv.heads;

        // rows before the first key that a tile sees
        for (int b = 0; b < a.batch; ++b) {
            const Extent e = extent_of(a, b);
            const int rows = e.qn * a.group;
            for (int tile = 0; tile < p.tiles; ++tile) {
                const int r0 = tile * p.rows_per_tile, r1 = std::min(rows, r0 + p.rows_per_tile);
                if (r0 >= rows)
                    continue;
                int lo, hi, least = 0x7FFFFFFF, end = 0;
                tile_keys(a, e, r0, r1, lo, hi);
                const int first = first_seen(a, e, r0);
                CHECK(lo == (first & ~31) && first - lo < kTileKeys && first <= std::max(hi, 0));
                for (int r = r0; r < r1; ++r) {
                    int s0, s1;
                    seen_by(a, e, r / a.group, s0, s1);
                    CHECK(s1 <= hi && s0 >= first);
                    if (s0 < s1) {
                        CHECK(end == 0 || s0 <= end); // without gaps: every other key of the tile is seen
                        least = std::min(least, s0);
                        end = std::max(end, s1);
                    }
                }
                CHECK(least == 0x7FFFFFFF || (least == first && end == hi));
                windows += first > lo;
            }
        }

        if (p.many) {
            int seen = 0;
            for (int b = 0; b < a.batch; ++b) {
                const Extent e = extent_of(a, b);
                const int rows = e.qn * a.group;
                for (int r0 = 0; r0 < rows; r0 += p.rows_per_tile) {
                    int lo, hi;
                    tile_keys(a, e, r0, std::min(rows, r0 + p.rows_per_tile), lo, hi);
                    const int n = chunks_of(p, lo, hi);
                    CHECK(n >= 1 && n <= p.chunks && (int64_t)n * p.chunk >= hi - lo);
                    seen = std::max(seen, n);
                }
            }
            most_chunks = std::max(most_chunks, seen);
            const size_t all = (size_t)pairs * a.max_q * a.group * p.chunks;
            CHECK(p.chunks == 1 || p.workspace == round256(all * 8) + all * a.kv.head_dim * 4);
            continue;
        }
        CHECK((p.chunks == 1) == (p.parts == 0));
        if (p.chunks == 1)
            continue;
        // the table, written and looked up as the kernels do
        const size_t bytes = few_table_bytes(p.groups, a.batch);
        CHECK((bytes != 0) == (a.batch > kScanBatch));
        uint32_t total = 0;
        for (int b = 0; b < a.batch; ++b)
            total += (uint32_t)few_steps(a, extent_of(a, b));
        const uint32_t most = few_most(p, total * a.kv.heads) + pick(0, 20); // the kernel may lengthen parts
        std::vector<uint32_t> space(bytes / 4 + 1);
        uint32_t parts_before = 0, slots_before = 0;
        FewTable t = few_table(space.data(), p.groups, a.batch);
        for (int b = 0; b < a.batch; ++b) {
            const uint32_t steps = few_steps(a, extent_of(a, b));
            const uint32_t parts = few_parts(steps, most), mine = parts * a.kv.heads;
            CHECK((steps == 0) == (parts == 0));
            if (bytes) {
                t.before[3 * b] = parts_before;
                t.before[3 * b + 1] = slots_before;
                t.before[3 * b + 2] = steps;
                for (uint32_t id = parts_before; id < parts_before + mine; ++id) {
                    CHECK(id < (uint32_t)p.groups);
                    t.sequence[id] = (uint32_t)b;
                }
            }
            int to = 0;
            for (uint32_t i = 0; i < parts; ++i) {
                CHECK(few_from(steps, parts, i) == to);
                to = few_from(steps, parts, i + 1);
                CHECK(to > few_from(steps, parts, i) && to - few_from(steps, parts, i) <= (int)most);
            }
            CHECK(to == (int)steps);
            parts_before += mine;
            slots_before += parts > 1 ? mine : 0;
        }
        CHECK(parts_before <= (uint32_t)p.groups && slots_before <= 2u * p.parts);
        if (bytes) {
            ++tables;
            *t.most = most;
            CHECK((char*)(t.most + 1) <= (char*)space.data() + bytes);
        }
        const size_t places = (size_t)2 * p.parts * p.rows_per_tile;
        CHECK(p.workspace == bytes + round256((size_t)pairs * 8) + round256(places * 8) + places * a.kv.head_dim * 4);
    }
    std::printf("%d tables, up to %d chunks, %d tiles with rows before their window\n", tables, most_chunks, windows);
    if (tables < 100 || most_chunks <= 64 || windows < 1000)
        return 1; // not what this is for
    std::printf("wide calls indexed clean\n");
    return 0;
}
