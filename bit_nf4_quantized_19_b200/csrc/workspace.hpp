// Scratch of one call, carved from the caller's workspace.  Host code only.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qlora {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Parts start on 256-byte addresses wherever the workspace itself starts (a caller's pointer is
// only 16-byte aligned, and kernels store up to 32 bytes at a time), so a workspace of 256 bytes
// more than its parts, each rounded up to 256, always holds them: what the size queries return.
struct Workspace {
  char *base;
  size_t used;
  size_t cap;
  void *take(size_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(base);
    const size_t off = align256(at + used) - at;
    if (off + bytes > cap) return nullptr;
    used = off + bytes;
    return base + off;
  }
};

}  // namespace qlora
