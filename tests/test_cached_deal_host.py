"""How attention over the paged cache deals its work out, on the host: the functions that the
kernels run (csrc/cattn_common.cuh) are compiled for the CPU and walked for every CTA of a
call.  Every block of every tile has to be worked on once, and every tile that several CTAs
share has to be announced to the kernel that joins the pieces: by the CTA that begins it,
however many tiles that CTA has."""
import math
import os
import random
import subprocess

import pytest

from channels_last_groupnorm_gb300 import build as gnbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "cattn_common.cuh"

using namespace gn::cattn;

struct Piece { int cta, b0, b1, at; };      // at: which of the CTA's segments

template <int K>
int walk(CattnArgs &a, int ctas, long long *shared_tiles, long long *at_a_list_end)
{
    const int n0 = first_sequence(a), n1 = n0 + sequence_count(a);
    std::vector<int64_t> units;
    int64_t all = 0, tiles = 0;
    for (int n = n0; n < n1; ++n) {
        Walk w(a);
        w.load(n);
        units.push_back(w.units());
        all += units.back();
        tiles += static_cast<int64_t>(w.runs) * w.heads();
    }
    const int busy = static_cast<int>(all < ctas ? (all > 0 ? all : 1) : ctas);
    std::map<std::tuple<int, int, int, int>, std::pair<int, std::vector<Piece>>> found;
    std::vector<Shared> words(ctas);
    for (int cta = 0; cta < ctas; ++cta) {
        Part part = {};
        if (cta < busy && all > 0) {
            const int64_t u0 = part_begin(all, busy, cta), u1 = part_begin(all, busy, cta + 1);
            int64_t before = 0;
            int n = 0;
            for (; n < n1 - n0 && before + units[n] <= u0; ++n) before += units[n];
            if (u0 < u1) part = {u0 - before, u1 - u0, u0, all, n0 + n, busy};
        }
        Walk w(a);
        w.start(part.seq, part.offset, part.count, part.first);
        static WorkList<K> list;
        words[cta] = {};
        for (int at = 0, more = 1; more;) {
            list_work(list, w, part, cta, words[cta]);
            for (int i = 0; i < list.count; ++i, ++at) {
                const Segment &g = list.list[i];
                if (g.b0 >= g.b1 || g.b1 > g.total || g.total != blocks_of(a, g.s, g.run)) return 1;
                auto &t = found[{g.seq, g.hk, g.first_head, g.run}];
                t.first = g.total;
                t.second.push_back({cta, g.b0, g.b1, at});
                if (g.b0 == 0 && g.b1 < g.total && (at + 1) % K == 0) ++*at_a_list_end;
            }
            more = list.more && list.count > 0;
        }
    }
    if (static_cast<int64_t>(found.size()) != tiles) return 2;
    int announced = 0;
    for (const Shared &s : words) announced += s.pieces != 0;
    for (const auto &f : found) {
        const auto &p = f.second.second;
        int at = 0;
        for (size_t i = 0; i < p.size(); ++i) {
            if (p[i].b0 != at || p[i].cta != p[0].cta + static_cast<int>(i)) return 3;
            if (i > 0 && p[i].at != 0) return 4;
            at = p[i].b1;
        }
        if (at != f.second.first) return 5;
        if (p.size() == 1) continue;
        ++*shared_tiles;
        --announced;
        const Shared &s = words[p[0].cta];
        const int seq = std::get<0>(f.first), hk = std::get<1>(f.first), head = std::get<2>(f.first), run = std::get<3>(f.first);
        const gn::cache::Sequence q = gn::cache::sequence_of(a.p.c, a.p.a.tokens, seq);
        if (s.pieces != static_cast<int>(p.size())) return 6;
        if (s.token != q.begin + run * a.tokens || s.head != hk * a.p.group + head || s.heads != a.p.group - head) return 7;
        if (s.rows != min(a.tokens, q.end - q.begin - run * a.tokens) * a.heads) return 8;
    }
    return announced == 0 ? 0 : 9;
}

int main()
{
    // per line: K ctas rows extra least most heads kv_heads page width causal given, lengths, new tokens ahead of, of and behind the sequences
    int k, ctas, rows, extra, least, most, heads, hk, page, width, causal, given, count, line = 0;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d", &k, &ctas, &rows, &extra, &least, &most, &heads, &hk, &page, &width,
                      &causal, &given, &count) == 13) {
        std::vector<int> lengths(count), cu(count + 1);
        int ahead, behind;
        for (int &v : lengths) if (std::scanf("%d", &v) != 1) return 2;
        if (std::scanf("%d", &ahead) != 1) return 2;
        cu[0] = ahead;
        for (int n = 0; n < count; ++n) {
            int v;
            if (std::scanf("%d", &v) != 1) return 2;
            cu[n + 1] = cu[n] + v;
        }
        if (std::scanf("%d", &behind) != 1) return 2;
        CattnArgs a = {};
        a.p.c.lengths = lengths.data();
        a.p.c.cu = given ? cu.data() : nullptr;
        a.p.c.table_width = width;
        a.p.c.page_size = page;
        a.p.c.sequences = count;
        a.p.c.kv_heads = hk;
        a.p.a.tokens = cu[count] + behind;
        a.p.a.heads = heads;
        a.p.a.causal = causal;
        a.p.group = heads / hk;
        a.least = least;
        a.most = most;
        a.extra = extra;
        a.rows = rows;
        a.heads = a.p.group < rows ? a.p.group : rows;
        a.chunks = (a.p.group + a.heads - 1) / a.heads;
        a.tokens = rows / a.heads;
        long long shared = 0, ends = 0;
        const int bad = k == 1    ? walk<1>(a, ctas, &shared, &ends)
                        : k == 2  ? walk<2>(a, ctas, &shared, &ends)
                        : k == 16 ? walk<16>(a, ctas, &shared, &ends)
                                  : walk<32>(a, ctas, &shared, &ends);
        std::printf("%d %d %lld %lld\n", line++, bad, shared, ends);
    }
}
"""

FEW = dict(k=32, ctas=304, rows=16, extra=4)          # of the kernel for few rows, and of the one for many
MANY = dict(k=16, ctas=152, rows=256, extra=8)
WHAT = {1: "a segment out of range", 2: "a tile that is missing", 3: "pieces that do not follow on one another",
        4: "a piece that is not its CTA's first", 5: "blocks that are missing", 6: "a shared tile that is not announced",
        7: "a shared tile announced elsewhere", 8: "its rows", 9: "a tile announced that is not shared"}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    to = tmp_path_factory.mktemp("deal")
    src, exe = to / "deal.cu", to / "deal"
    src.write_text(PROGRAM)
    csrc = os.path.join(gnbuild.HERE, "csrc")
    subprocess.run([gnbuild.nvcc(), *gnbuild.ARCH, "-O1", "-std=c++17", "-I", csrc, "-o", str(exe), str(src)], check=True,
                   capture_output=True)
    return str(exe)


def line(kernel, lens, new, heads, kv_heads, page=64, causal=True, given=True, ahead=0, behind=0, least=0, most=2 ** 31 - 1, width=None):
    width = width or max(1, max((n + page - 1) // page for n in lens))
    head = [kernel["k"], kernel["ctas"], kernel["rows"], kernel["extra"], least, most, heads, kv_heads, page, width, int(causal),
            int(given), len(lens)]
    return " ".join(map(str, head + list(lens) + [ahead] + list(new) + [behind]))


def run(program, lines):
    """Checks every call; how many shared tiles each has, and how many of them end a list."""
    r = subprocess.run([program], input="\n".join(lines) + "\n", text=True, check=True, capture_output=True)
    rows = [[int(v) for v in out.split()] for out in r.stdout.splitlines()]
    assert len(rows) == len(lines)
    for n, bad, _, _ in rows:
        assert bad == 0, f"{WHAT[bad]}: {lines[n][:300]}"
    return [(shared, ends) for _, _, shared, ends in rows]


@pytest.mark.parametrize("kernel,lens,new,heads,kv_heads", [
    (MANY, [12288], [12288], 32, 8), (MANY, [10000], [10000], 32, 8), (MANY, [32768], [32768], 32, 8), (MANY, [8192], [8192], 64, 8),
    (MANY, [2048] * 8, [2048] * 8, 32, 8), (MANY, [2000] * 290, [64] * 290, 32, 8), (FEW, [4096] * 296, [1] * 296, 32, 32),
    (FEW, [4096] * 1180, [1] * 1180, 32, 8), (FEW, [1000] * 1180, [1] * 1180, 32, 8)])
def test_shared_tiles_that_end_a_list(program, kernel, lens, new, heads, kv_heads):
    found = run(program, [line(kernel, lens, new, heads, kv_heads)])
    assert found[0][1] > 0            # (what this test is for)


def test_draws_of_lengths(program):
    rng, lines = random.Random(7), []

    def log(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    for _ in range(400):
        kernel = dict(rng.choice([FEW, MANY]))
        kernel["k"] = rng.choice([1, 2, kernel["k"], kernel["k"]])
        kernel["ctas"] = rng.choice([kernel["ctas"], kernel["ctas"], log(1, 400)])
        kv_heads = rng.choice([1, 2, 3, 8, 32])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 17])
        count = log(1, 400 if kv_heads < 32 else 100)
        given = rng.random() < 0.7
        most = log(1, 40) if kernel["rows"] == 16 else log(1, 4000 // count + 1)
        new = [rng.choice([1, most, rng.randint(0, most)]) for _ in range(count)] if given else [rng.randint(1, most)] * count
        lens = [rng.choice([n, n + rng.randint(0, 300), rng.randint(0, 10), log(16, 16384)]) for n in new]
        least = rng.choice([0, 0, 2]) if given else 0
        lines.append(line(kernel, lens, new, heads, kv_heads, page=rng.choice([8, 24, 64, 256]), causal=rng.random() < 0.8, given=given,
                          ahead=rng.choice([0, 3, 700]) if given else 0, behind=rng.choice([0, 5, 300]) if given else 0, least=least,
                          most=rng.choice([2 ** 31 - 1, least + most // 2]) if given else 2 ** 31 - 1,
                          width=rng.choice([None, None, 20])))
    found = run(program, lines)
    assert sum(s for s, _ in found) > 1000 and sum(e for _, e in found) > 100
