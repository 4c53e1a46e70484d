"""The page selection's search by groups of 16 pages, on the host: the rule that admits
it is the kernel's own, compiled from csrc/select_groups.cuh; the search itself is walked
as page_select.cu does it, in its integer arithmetic, against a sort."""
import ctypes
import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_frequency_sparse_b200", "csrc")

# Every (pages, n_first, n_last, n_select) up to `most` pages, and windows of 128 to 1024
# first or last pages around the lengths where few groups compete.  The kernel takes the
# scores' threshold from the places-th highest group among those that hold a competing
# page: where it searches, there must be that many of them, and it must look at each.
RULE = r"""
#include <cstdio>
#include <cstdlib>
#include "select_groups.cuh"
static long searched = 0;
static void check(int pages, int first, int last, int n_select) {
  const int places = n_select - first - last;
  if (places < 1 || pages <= n_select) return;  // answered before the search
  const atf::SelectGroups g = atf::select_groups(pages, first, last, places);
  if (!g.search) return;
  ++searched;
  int rivals = 0, lowest = -1, highest = -1;
  for (int k = 0; k * atf::kGroup < pages; ++k) {
    bool competes = false;
    for (int i = k * atf::kGroup; i < (k + 1) * atf::kGroup && i < pages; ++i) competes |= i >= first && i < pages - last;
    if (competes) lowest = lowest < 0 ? k : lowest, highest = k, ++rivals;
  }
  if (rivals < places || g.first != lowest || g.count != rivals || highest != lowest + rivals - 1) {
    std::printf("%d pages, first %d, last %d, select %d: %d places, %d competing groups from %d, searched %d from %d\n",
                pages, first, last, n_select, places, rivals, lowest, g.count, g.first);
    std::exit(1);
  }
}
int main() {
  const int most = 100;
  for (int pages = 1; pages <= most; ++pages)
    for (int first = 0; first < pages; ++first)
      for (int last = 0; first + last < pages; ++last)
        for (int n = first + last + 1; n < pages; ++n) check(pages, first, last, n);
  const int windows[] = {110, 128, 256, 512, 1000, 1024};
  for (int w : windows)
    for (int other = 0; other < 20; ++other)
      for (int places = 1; places < 40; ++places)
        for (int pages = w; pages < w + 1200; ++pages) {
          check(pages, other, w, other + w + places);
          check(pages, w, other, other + w + places);
        }
  std::printf("searched %ld\n", searched);
  return searched ? 0 : 1;
}
"""


def test_searched_groups_hold_as_many_rivals_as_places(tmp_path):
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(RULE)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I" + CSRC, str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


# ------------------------------------------------------------------ the search, walked

SOURCE = open(os.path.join(CSRC, "page_select.cu")).read()
BINS, BIN_BITS = (int(x) for x in re.search(r"kBins = (\d+), kBinBits = (\d+);", SOURCE).groups())
AGAIN, CANDIDATES, FEW_GROUPS = (int(re.search(rf"{n} = (\d+);", SOURCE).group(1))
                                 for n in ("kAgain", "kCandidates", "kFewGroups"))
GROUP = 16


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    where = tmp_path_factory.mktemp("rule")
    src, lib = where / "rule.cpp", where / "rule.so"
    src.write_text('#include "select_groups.cuh"\n'
                   'extern "C" void rule(int pages, int first, int last, int places, int* out) {\n'
                   "  const atf::SelectGroups g = atf::select_groups(pages, first, last, places);\n"
                   "  out[0] = g.first, out[1] = g.count, out[2] = g.search;\n}\n")
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(lib)])
    fn = ctypes.CDLL(str(lib)).rule

    def call(*args):
        out = (ctypes.c_int * 3)()
        fn(*args, out)
        return list(out)

    return call


# what a round leaves where no bin holds the rank: the state that one thread sets beforehand
PRESET = re.search(r"if \(tid == 0\) sh->lo = sh->hi = lo, sh->need = need, sh->count = count;", SOURCE) is not None


def _narrow(keys, lo, hi, need, count, few, bits=32, held=True):
    """[lo, hi] narrowed to the bin of the need-th highest key, round by round; held: the keys hold that rank."""
    rounds = 0
    while lo < hi and count > few and count != need:
        shift = max(0, (hi - lo).bit_length() - BIN_BITS)
        hist = [0] * BINS
        for k in keys:
            if lo <= k <= hi:
                hist[(k - lo) >> shift] += 1
        before, found = 0, None
        for b in reversed(range(BINS)):
            if before < need <= before + hist[b]:
                found = b
                break
            before += hist[b]
        assert found is not None or not held, "a rank that no bin holds"
        if found is None:
            assert PRESET, "a round that reads what nobody wrote"
            hi = lo
            continue
        lo = lo + (found << shift)
        hi = min(hi, lo + (1 << shift) - 1)
        need, count = need - before, hist[found]
        rounds += 1
        assert rounds <= -(-bits // BIN_BITS)
    return lo, hi, need, count


def _search(rule, score, first, last, n_select, slack):
    """The kept competing pages by the search over groups (None: it passes the list on).  score: the scores of
    the pages in 64 bits; the 32-bit ones are off by up to slack / 2."""
    pages, places = len(score), n_select - first - last
    g0, count, search = rule(pages, first, last, places)
    if not search:
        return None
    r = random.Random(pages)
    key = [s + r.randint(-(slack // 2), slack // 2) for s in score]
    groups = range(g0, g0 + count)
    # a group's highest competing score; 0 where it has none
    high = {k: max([key[i] for i in range(k * GROUP, (k + 1) * GROUP) if first <= i < pages - last], default=0)
            for k in groups}
    assert min(high.values()) > 0 and len(high) >= places
    top = max(high.values())
    lo, *_ = _narrow(high.values(), min(high.values()), top, places, count, FEW_GROUPS)
    least = lo - slack
    kept_groups = [k for k in groups if high[k] >= least]
    if len(kept_groups) > CANDIDATES // GROUP:
        return None
    cand = [i for k in kept_groups for i in range(k * GROUP, min(pages, (k + 1) * GROUP))
            if first <= i < pages - last and key[i] >= least]
    lo, hi, *_ = _narrow([key[i] for i in cand], least, top, places, len(cand), 1)
    above = [i for i in cand if key[i] > hi + slack]
    close = [i for i in cand if lo - slack <= key[i] <= hi + slack]
    if len(close) > AGAIN:
        return None
    need = places - len(above)
    return sorted(above + sorted(close, key=lambda i: (-score[i], i))[:need])


@pytest.mark.parametrize("seed", range(60))
def test_search_over_groups_is_a_sort(rule, seed):
    r = random.Random(seed)
    searched = 0
    for _ in range(60):
        places = r.choice([1, 1, 2, 3, 5, 8, 40])
        first, last = r.choice([(1, 1), (0, 0), (1, 110), (1, 128), (1, 256), (1, 512), (128, 3), (600, 2),
                                (r.randint(0, 200), r.randint(0, 200))])
        n = first + last + places
        pages = n + r.choice([1, r.randint(1, 40), r.randint(1, 2500)])
        wide = r.choice([3, 1000, 1 << 30])
        score = [(1 << 29) + r.randrange(wide) for _ in range(pages)]
        got = _search(rule, score, first, last, n, r.choice([0, 0, 2, 100]))
        if got is None:
            continue
        searched += 1
        want = sorted(range(first, pages - last), key=lambda i: (-score[i], i))[:places]
        assert got == sorted(want), (pages, first, last, n)
    assert searched


@pytest.mark.parametrize("seed", range(40))
def test_narrowing_ends_whatever_it_is_given(seed):
    """Ranks that the keys do not hold, counts that are not theirs, keys outside the range."""
    r = random.Random(seed)
    for _ in range(20):
        bits = r.choice([32, 64])
        keys = [r.randrange(1 << r.randint(1, bits)) for _ in range(r.choice([0, 1, 5, 300]))]
        lo, hi = sorted(r.randrange(1 << r.randint(1, bits)) for _ in range(2))
        _narrow(keys, lo, hi, r.randint(0, 2 * len(keys) + 2), r.randint(0, 2 * len(keys) + 2), r.choice([1, 24]), bits,
                held=False)
