// Parts of a workspace at every start that is a multiple of 16: 256-byte addresses, no overlap, none
// past the end, all of them held by 256 bytes more than their rounded sizes, and refused by less
// than they need.  Prints the number of checks; the first failure ends it.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "workspace.hpp"

static long checks = 0;
static void check(bool ok, const char *what, size_t start, size_t i) {
  ++checks;
  if (ok) return;
  printf("failed: %s (start %zu, part %zu)\n", what, start, i);
  exit(1);
}

int main() {
  const size_t lists[][6] = {
      {1, 16, 255, 256, 257, 4096}, {4096, 32, 0, 48, 4000, 16}, {0, 0, 24, 512, 8, 1000}, {300, 300, 300, 300, 300, 300}};
  char *mem = static_cast<char *>(aligned_alloc(256, 1 << 16));
  for (const auto &sizes : lists) {
    size_t query = 256, plain = 0;
    for (size_t s : sizes) {
      query += qlora::align256(s);
      plain += s;
    }
    for (size_t start = 0; start < 512; start += 16) {
      qlora::Workspace ws{mem + start, 0, query};
      char *end = mem + start;
      for (size_t i = 0; i < 6; ++i) {
        char *p = static_cast<char *>(ws.take(sizes[i]));
        check(p != nullptr, "a part does not fit into the size the query returns", start, i);
        check(reinterpret_cast<uintptr_t>(p) % 256 == 0, "a part is not on a 256-byte address", start, i);
        check(p >= end && p + sizes[i] <= mem + start + query, "a part overlaps or leaves the workspace", start, i);
        end = p + sizes[i];
      }
      qlora::Workspace small{mem + start, 0, plain - 1};
      bool refused = false;
      for (size_t s : sizes) refused = refused || small.take(s) == nullptr;
      check(refused, "a workspace smaller than its parts is taken", start, 0);
    }
  }
  free(mem);
  printf("%ld checks\n", checks);
  return 0;
}
