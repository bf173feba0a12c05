// per_device.h on the host: a number is found out once for each device, a failure is
// not kept, and devices past the table are asked every time.
#include <stdio.h>
#include <string.h>

#include "per_device.h"

static int calls[200];
static int current;

static int number(dkv::PerDevice& known, int dev, int* out, int fail) {
  current = dev;
  return dkv::per_device(known, dev, 0, out, [fail](int* n) {
    ++calls[current];
    *n = fail ? 0 : 100 + current;
    return fail;
  });
}

#define CHECK(x) \
  if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1

int main() {
  static dkv::PerDevice known, other;
  int n = 0;
  for (int turn = 0; turn < 3; ++turn)
    for (int dev = 0; dev < dkv::kMaxDevices; ++dev) {
      CHECK(number(known, dev, &n, 0) == 0 && n == 100 + dev);
      CHECK(calls[dev] == 1);
    }
  for (int turn = 1; turn < 4; ++turn) {
    CHECK(number(known, 150, &n, 0) == 0 && n == 250);
    CHECK(calls[150] == turn);
  }
  memset(calls, 0, sizeof calls);
  n = -5;
  CHECK(number(other, 3, &n, 7) == 7 && n == -5);
  CHECK(number(other, 3, &n, 0) == 0 && n == 103 && calls[3] == 2);
  CHECK(number(other, 3, &n, 7) == 0 && n == 103 && calls[3] == 2);
  return 0;
}
