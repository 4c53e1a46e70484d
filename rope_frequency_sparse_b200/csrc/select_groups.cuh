// select_groups.cuh -- which groups of pages a page selection searches by their highest
// scores.  Plain constexpr C++: the kernel and a host check compile it.
#pragma once

namespace atf {

constexpr int kGroup = 16;  // pages of a group

// Pages [n_first, pages - n_last) compete for `places`; the others are kept anyway.
struct SelectGroups {
  int first, count;  // the groups that hold a competing page
  bool search;       // whether they are searched before the pages are
};

// Places below 1 or nothing to choose (pages - n_first - n_last <= places) do not come here.
// A group of forced pages alone has no score, so only the others count: the search takes its
// threshold from the places-th highest of them, and each of `places` groups then holds a
// candidate.  Four groups a place: fewer leave the pages of most groups to be looked at.
constexpr SelectGroups select_groups(int pages, int n_first, int n_last, int places) {
  const int first = n_first / kGroup, count = (pages - n_last - 1) / kGroup - first + 1;
  return {first, count, count >= 4 * places};
}

}  // namespace atf
