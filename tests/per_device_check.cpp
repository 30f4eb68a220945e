// Host-side check of answers kept for each device (per_device.h), with fake
// devices: none gets another's answer, each question is asked once, one that
// failed is asked again, and devices beyond the table are asked every time.
// Prints one line; exit code 0 when all pass.
#include <cstdio>

#include "per_device.h"

using namespace ep;

static PerDevice<3> known;
static int asked = 0;

static int get(int device, int kind, bool fails = false) {
    return known.get(device, kind, 1, [&](int* n) {
        ++asked;
        *n = fails ? 0 : 100 * (device + 1) + kind;
        return !fails;
    });
}

int main() {
    int wrong = 0;
    auto want = [&](const char* what, int got, int value, int asks) {
        if (got == value && asked == asks) return;
        ++wrong;
        std::printf("%s: %d asked %d times, not %d asked %d times\n", what, got, asked, value, asks);
    };
    want("first", get(0, 0), 100, 1);
    want("known", get(0, 0), 100, 1);
    want("another question", get(0, 2), 102, 2);
    want("another device", get(1, 0), 200, 3);
    want("the first again", get(0, 0), 100, 3);
    want("a failure", get(2, 1, true), 1, 4);
    want("after a failure", get(2, 1), 301, 5);
    want("known after it", get(2, 1, true), 301, 5);
    want("past the table", get(kKnownDevices, 0), 100 * (kKnownDevices + 1), 6);
    want("past the table again", get(kKnownDevices, 0), 100 * (kKnownDevices + 1), 7);
    want("no device", get(-1, 0, true), 1, 8);
    if (wrong > 0) return 1;
    std::printf("per device ok\n");
    return 0;
}
