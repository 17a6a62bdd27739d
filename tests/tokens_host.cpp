// The host-made arguments of the kernels on token rows, checked on the CPU:
// quotients, the cut of a sort into workgroups, and the page and place of a
// token, which the kernels compute with the same functions.
#include <stdio.h>

#include "../bmmc_affine_index_amd/csrc/tokens/tokens.h"

using namespace bmmc;

static int bad = 0;
#define CHECK(x)                                             \
    do {                                                     \
        if (!(x)) {                                          \
            printf("failed at %d: %s\n", __LINE__, #x);      \
            ++bad;                                           \
        }                                                    \
    } while (0)

static void quotients() {
    const uint32_t most = 0x7fffffffu;
    for (uint32_t d = 1; d < 3000; ++d) {
        const FastDiv f = fast_div(d);
        for (uint32_t n = 0; n < 5000; n += 7) CHECK(quotient(f, n) == n / d);
        for (uint32_t k = 0; k < 40; ++k) {
            const uint32_t n = most - k * 53693u;
            CHECK(quotient(f, n) == n / d);
            const uint32_t m = n / d * d;  // the borders, where a wrong factor shows
            CHECK(quotient(f, m) == m / d);
            if (m) CHECK(quotient(f, m - 1) == (m - 1) / d);
        }
    }
    const uint32_t wide[] = {65535, 65536, 65537, 1u << 24, (1u << 30) + 1, most - 1, most};
    for (uint32_t d : wide) {
        const FastDiv f = fast_div(d);
        for (uint32_t k = 0; k < 3000; ++k) CHECK(quotient(f, most - k) == (most - k) / d);
        CHECK(quotient(f, d - 1) == 0 && quotient(f, d) == 1);
    }
}

static void cuts() {
    const int64_t counts[] = {0, 1, 63, 64, 4095, 4096, 4097, 8192, 131072, 524287, 524288, 524289,
                              1 << 20, (int64_t(1) << 31) - 1};
    for (int64_t n : counts) {
        const OrderCut c = order_cut(n);
        CHECK(c.blocks >= 1 && c.blocks <= kOrderMaxBlocks);
        CHECK(c.chunk * c.blocks >= n);
        CHECK(c.blocks == 1 || c.chunk * (c.blocks - 1) < n);
        CHECK(c.blocks == 1 || c.chunk % 64 == 0);
    }
}

static void places() {
    const int32_t table[] = {5, 2, -1, 7,  // sequence 0 (a row of 4, of which 3 are the table's)
                             0, 9, 3, 7};
    const int32_t seqs[] = {0, 0, 0, 1, 1, -1, 2, 0, 1};
    const int32_t pos[] = {0, 17, 32, 15, 16, 0, 0, -1, 48};
    PageTable t{table, seqs, pos, 2, 3, 4, 8, 16, 0};
    const int32_t page[] = {5, 2, -1, 0, -1, -1, -1, -1, -1};
    const int32_t place[] = {0, 1, 0, 15};
    for (int i = 0; i < 9; ++i) CHECK(page_place(t, i).page == page[i]);
    for (int i = 0; i < 4; ++i) CHECK(page[i] < 0 || page_place(t, i).place == place[i]);
    // without sequences token t is sequence t's; past the batch it is nowhere
    t.sequences = nullptr;
    CHECK(page_place(t, 0).page == 5 && page_place(t, 1).page == 9 - 9 - 1);  // 9 >= 8 pages
    CHECK(page_place(t, 2).page == -1);
    // positions past 32 bits, pages of odd sizes
    const int64_t far[] = {(int64_t(1) << 31) + 5, (int64_t(1) << 62), (int64_t)-1 << 40, 14};
    t.positions = far;
    t.positions_are_64 = 1;
    t.batch = 2;
    const int32_t zero[] = {0, 0, 0, 1};
    t.sequences = zero;
    for (int i = 0; i < 3; ++i) CHECK(page_place(t, i).page == -1);
    t.page_size = 7;
    CHECK(page_place(t, 3).page == 3 && page_place(t, 3).place == 0);
    t.page_size = (int64_t(1) << 31) - 1;  // one page as long as they come
    const PagePlace p = page_place(t, 0);
    CHECK(p.page == 2 && p.place == 6);
    t.batch = 0;
    CHECK(page_place(t, 3).page == -1);
}

int main() {
    quotients();
    cuts();
    places();
    printf("%s\n", bad ? "FAILED" : "ok");
    return bad != 0;
}
