/* Host helpers of the library that need no device: an answer of the runtime is
 * kept, a failure to answer is not.  Exit status 0 on success. */
#include <stdio.h>

#include "gnq_host.cuh"

static int fail(const char *what) {
    fprintf(stderr, "FAIL: %s\n", what);
    return 1;
}

int main() {
    std::atomic<int> slot{0};
    int asked = 0;
    if (gnq::answer_once(slot, [&] { ++asked; return -1; }) != -1) return fail("a failure is reported");
    if (gnq::answer_once(slot, [&] { ++asked; return 23; }) != 23) return fail("a failure was kept");
    if (gnq::answer_once(slot, [&] { ++asked; return 7; }) != 23 || asked != 2) return fail("an answer was not kept");
    std::atomic<int> none{0};
    if (gnq::answer_once(none, [&] { ++asked; return 0; }) != 0) return fail("0 is an answer");
    if (gnq::answer_once(none, [&] { ++asked; return 1; }) != 0 || asked != 3) return fail("0 was not kept");
    printf("host helpers ok\n");
    return 0;
}
