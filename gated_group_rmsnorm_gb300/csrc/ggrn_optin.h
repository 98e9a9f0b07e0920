// ggrn_optin.h -- kernels' opt-in to more than 48 KB of dynamic shared memory.
// The attribute belongs to a kernel on one device, so it is set once for each
// device that launches the kernel.
#pragma once

namespace ggrn {

// Runs set() unless it has succeeded before for device `dev` under this word
// (a bit per device; devices past the word's bits run it every time).  set()
// returns 0 for success; another status is returned and not remembered.  Two
// threads may both run it.
template <typename Set>
auto once_per_device(unsigned long long* done, int dev, Set set) -> decltype(set()) {
  using Status = decltype(set());
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (__atomic_load_n(done, __ATOMIC_ACQUIRE) & bit) return Status{};
  const Status st = set();
  if (st == Status{}) __atomic_fetch_or(done, bit, __ATOMIC_RELEASE);
  return st;
}

#ifdef __CUDACC__
// A template on the kernel itself: every instantiation has a word of its own.
template <auto kernel>
cudaError_t allow_shared_memory(int bytes) {
  static unsigned long long done = 0;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once_per_device(&done, dev, [bytes] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}
#endif

}  // namespace ggrn
