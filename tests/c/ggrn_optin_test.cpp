// Host test of the rule that sets a kernel's shared-memory limit once for each
// device (gated_group_rmsnorm_gb300/csrc/ggrn_optin.h): the tests build it with
// the host C++ compiler and run it.  Devices and the call that sets the limit
// are the test's own.
#include <cstdio>

#include "ggrn_optin.h"

namespace {

int failures = 0;
void expect(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAIL %s\n", what);
    ++failures;
  }
}

int calls[80];
int status = 0;
unsigned long long word = 0;

int launch(int dev) {
  return ggrn::once_per_device(&word, dev, [dev] {
    ++calls[dev];
    return status;
  });
}

}  // namespace

int main() {
  expect(launch(0) == 0 && calls[0] == 1, "the first launch sets the limit");
  expect(launch(0) == 0 && calls[0] == 1, "the second one need not");
  expect(launch(1) == 0 && calls[1] == 1, "another device needs its own");
  expect(launch(63) == 0 && calls[63] == 1 && launch(63) == 0 && calls[63] == 1, "the last bit");
  expect(launch(0) == 0 && launch(1) == 0 && calls[0] == 1 && calls[1] == 1, "all are remembered");
  status = 7;
  expect(launch(2) == 7 && calls[2] == 1, "a failure is returned");
  expect(launch(2) == 7 && calls[2] == 2, "and tried again");
  expect(launch(0) == 0, "other devices keep theirs");
  status = 0;
  expect(launch(2) == 0 && calls[2] == 3 && launch(2) == 0 && calls[2] == 3, "until it succeeds");
  expect(launch(64) == 0 && launch(64) == 0 && calls[64] == 2, "devices past the word");
  unsigned long long other = 0;
  int n = 0;
  ggrn::once_per_device(&other, 0, [&n] { return ++n, 0; });
  expect(n == 1, "another kernel's word is its own");
  std::printf("failures %d\n", failures);
  return failures != 0;
}
