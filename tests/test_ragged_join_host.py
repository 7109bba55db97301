"""Which block of the merge joins which part of which token, on a machine without
a GPU: the kernels' own cut and assignment, compiled for the host."""

import random
import subprocess

import pytest

from mla_latent_kv_39_b200 import build

# Reads cases "window sinks batch workers, cu_q.., seq_lens..", all fine, and prints
# per case, for every token that several workers hold: token, workers from the first to
# the last, and the least and the greatest number of times that one of its half heads is
# joined; then how many joins went to anything else.
PROGRAM = r'''
#include <algorithm>
#include <cstdio>
#include <map>
#include <vector>
#include "chunk_plan.cuh"
using namespace mla::chunk;
int main() {
  const int heads = 128;
  int window, sinks, batch, workers;
  while (std::scanf("%d %d %d %d", &window, &sinks, &batch, &workers) == 4) {
    std::vector<int32_t> cu(batch + 1), len(batch);
    for (auto& x : cu) std::scanf("%d", &x);
    for (auto& x : len) std::scanf("%d", &x);
    const Batch q{cu.data(), len.data(), batch, cu[batch], 1 << 20, Visible{window, sinks}};
    Cut cut{0, workers, 1.f / workers, 0};
    long long tokens = 0, longest = 0;
    for (int b = 0; b < batch; ++b) {
      const Sequence s = sequence_of(q, b);
      cut.total += cut.tokens(q.vis, s, s.n);
      tokens += s.n;
      longest = std::max(longest, longest_token(q.vis, s));
    }
    if (one_token_each(tokens, cut.total, longest, workers)) {
      cut.single = 1;
      cut.total = tokens;
    }
    std::vector<long long> C(batch + 1, 0);
    for (int b = 0; b < batch; ++b) {
      const Sequence s = sequence_of(q, b);
      C[b + 1] = C[b] + cut.tokens(q.vis, s, s.n);
    }
    struct Held { int first, last, parts; };
    std::map<int, Held> held;
    std::vector<Shares> shares(workers);
    for (int w = 0; w < workers; ++w) {
      const Found from = place_at(q, cut, C.data(), cut.at(w)), to = place_at(q, cut, C.data(), cut.at(w + 1));
      shares[w] = shares_of(q, cut, from, to, w);
      for (Walk k(q, from.at, from.s, to.at); k.valid(); k.next()) {
        auto it = held.emplace(k.token(), Held{w, w, 0}).first;
        it->second.last = w;
        ++it->second.parts;
      }
    }
    // the joins of every block, counted by half heads
    std::map<int, std::vector<int>> joined;
    long long stray = 0;
    for (int w = 0; w < workers; ++w) {
      const Join j = join_of(shares.data(), w);
      if (j.token < 0) continue;
      const auto it = held.find(j.token);
      const bool fine = it != held.end() && it->second.parts > 1 && it->second.first == j.first &&
                        it->second.last == j.first + j.n - 1;
      auto& n = joined[j.token];
      n.resize(2 * heads, 0);
      for (int y = 0; y < kMergeY; ++y)
        for (int i = j.begin(w, y); i < j.items(heads); i += j.step()) {
          if (!fine) ++stray;
          if (j.many()) ++n[i];
          else for (int h = 8 * i; h < 8 * i + 8; ++h) ++n[h];
        }
    }
    std::printf("case\n");
    for (const auto& t : held) {
      if (t.second.parts < 2) continue;
      auto& n = joined[t.first];
      n.resize(2 * heads, 0);
      std::printf("token %d %d %d %d\n", t.first, t.second.last - t.second.first + 1, *std::min_element(n.begin(), n.end()),
                  *std::max_element(n.begin(), n.end()));
    }
    std::printf("stray %lld\n", stray);
  }
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    (d / "join.cu").write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH_FLAGS, "-std=c++17", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o",
                    str(d / "join"), str(d / "join.cu")], check=True, capture_output=True)
    return d / "join"


def joins(program, cases):
    """Per case the split tokens as (token, workers, least, greatest) and the stray joins."""
    lines = []
    for window, sinks, cached, new, workers in cases:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        lines.append(" ".join(map(str, [window, sinks, len(new), workers] + cu + [c + n for c, n in zip(cached, new)])))
    out = subprocess.run([str(program)], input="\n".join(lines), capture_output=True, text=True, check=True).stdout
    got = []
    for block in out.split("case\n")[1:]:
        rows = [ln.split() for ln in block.splitlines()]
        got.append(([tuple(map(int, r[1:])) for r in rows if r[0] == "token"], int(rows[-1][1])))
    assert len(got) == len(cases)
    return got


def random_cases(n, seed):
    r = random.Random(seed)
    cases = []
    for _ in range(n):
        kind = r.choice(["decode", "decode", "chunks", "mixed", "window", "equal"])
        batch = r.choice([1, 2, 3, 4, 5, 6, 8, 12, 16, 20, 40])
        new = [1] * batch
        cached = [r.randint(2000, 100000) for _ in range(batch)]
        window = sinks = 0
        if kind == "equal":
            cached = [r.choice([8001, 10000, 16383, 16384, 50000])] * batch
        elif kind == "chunks":
            new = [r.randint(0, 10) for _ in range(batch)]
        elif kind == "mixed":
            new = [r.choice([0, 1, 1, 2, 300]) for _ in range(batch)]
            cached = [r.choice([0, 64, 700, 9000, 16000, 60000]) for _ in range(batch)]
        elif kind == "window":
            window, sinks = r.choice([(8192, 4), (4000, 0), (20000, 130), (1000, 70)])
        cases.append((window, sinks, cached, new, r.choice([74, 74, 74, 73, 37, 20, 9, 2])))
    return cases


NAMED = [
    (0, 0, [10000] * 6, [1] * 6, 74), (0, 0, [10000, 10000, 10000, 2000], [1] * 4, 74), (0, 0, [16384] * 4, [1] * 4, 74),
    (0, 0, [100000] * 8, [1] * 8, 74), (0, 0, [8000, 20000, 3000, 16000], [1] * 4, 74), (0, 0, [16384] * 2, [4] * 2, 74),
    (8192, 4, [16384] * 5, [1] * 5, 74), (0, 0, [16000], [3], 74), (0, 0, [16000], [10], 74),
    (0, 0, [40000, 0, 30000], [1, 200, 1], 74)]


@pytest.mark.parametrize("cases", [NAMED, random_cases(3000, 1)], ids=["named", "random"])
def test_every_half_head_of_a_split_token_is_joined_once(program, cases):
    seen = set()
    for case, (tokens, stray) in zip(cases, joins(program, cases)):
        assert stray == 0, case
        for token, workers, least, greatest in tokens:
            assert (least, greatest) == (1, 1), (case, token, workers)
            seen.add(workers)
    if cases is not NAMED:      # tokens of few pieces, of many, and of more than can help
        assert {2, 8, 9, 10, 20, 31, 32, 33, 40, 74} <= seen
