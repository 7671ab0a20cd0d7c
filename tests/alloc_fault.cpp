// operator new for a preloaded object: fails the n-th allocation of at least
// `bytes` after fail_allocation(n, bytes) (n = 0: the next one), once.
#include <cstdlib>
#include <new>

namespace {
long left = -1;
std::size_t least = 0;
}  // namespace

extern "C" void fail_allocation(long n, std::size_t bytes) {
  left = n;
  least = bytes;
}
// Whether the failure is still to come; ends the wait for it.
extern "C" int allocation_fault_pending() {
  const int pending = left >= 0;
  left = -1;
  return pending;
}

void* operator new(std::size_t n) {
  if (left >= 0 && n >= least && left-- == 0) throw std::bad_alloc();
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
