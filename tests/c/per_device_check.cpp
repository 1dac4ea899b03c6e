// What the library keeps for each device (PerDevice of fp8bq_internal.h), with
// the two CUDA calls it makes replaced by these.
#include <cstdio>

#include "fp8bq_internal.h"

static int device = 0;
extern "C" cudaError_t cudaGetDevice(int *d) {
    *d = device;
    return cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError(void) { return cudaSuccess; }

#define CHECK(c) \
    if (!(c)) return std::fprintf(stderr, "line %d: %s\n", __LINE__, #c), 1

int main() {
    int made = 0, value = -1;
    auto make = [&] { return ++made, value; };
    auto good = [](int v) { return v >= 0; };
    static fp8bq::PerDevice<int> p;
    CHECK(p.get(make, good) == -1 && p.get(make, good) == -1 && made == 2);  // failures are not kept
    value = 7;
    CHECK(p.get(make, good) == 7 && made == 3);
    value = 8;
    CHECK(p.get(make, good) == 7 && made == 3);  // a success is
    device = 1;
    CHECK(p.get(make, good) == 8 && made == 4);  // each device its own
    device = 0;
    CHECK(p.get(make, good) == 7 && made == 4);
    device = fp8bq::kMaxDevices;
    CHECK(p.get(make, good) == 8 && p.get(make, good) == 8 && made == 6);
    device = 0;
    static fp8bq::PerDevice<int> all;
    value = -1;
    CHECK(all.get(make) == -1);
    value = 3;
    CHECK(all.get(make) == -1);  // without a test everything is kept
    std::puts("per device ok");
    return 0;
}
