// Host check of the sizes that csrc/gemm_validate.hpp plans for adapters, weight gradients
// from packed activations and the balance loss, built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_plan_cpu.py: parts that cover their tokens,
// workspaces that hold what the kernels write, and the extreme sizes where the arithmetic
// could overflow.  Prints one line per failure and exits nonzero.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "gemm_validate.hpp"

using namespace libgemm_host;

static int g_fail = 0, g_checked = 0;

#define CHECK(what)                                                              \
    do {                                                                         \
        ++g_checked;                                                             \
        if (!(what)) {                                                           \
            printf("FAIL line %d: %s (%lld %lld %lld)\n", __LINE__, #what, (long long)a, (long long)b, (long long)c); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

static const void *P(uint64_t a) { return reinterpret_cast<const void *>((uintptr_t)a); }

static void wgrad(int64_t a, int64_t b, int64_t c) {
    const WgradPlan w = wgrad_plan(a, b, c);
    CHECK(w.bm == 32 || w.bm == 64 || w.bm == 128 || w.bm == 256);
    CHECK(w.bn == 128 || w.bn == 256);
    CHECK(b > 64 || b <= w.bm);  // thin: one tile
    CHECK(w.per > 0 && w.per % 64 == 0 && w.splits >= 1 && w.splits <= 64);
    CHECK(w.splits * w.per >= a);              // every token has a part
    CHECK(w.splits == 1 || (w.splits - 1) * w.per < a);  // no part is empty
    CHECK(w.per < (int64_t)1 << 32);
    const int64_t bytes = checkpoint_wgrad_workspace(a, b, c);
    const __int128 sums = (__int128)w.splits * b * ((c + 3) / 4 * 4) * 4;
    CHECK(w.splits == 1 ? bytes == 0 : (__int128)bytes >= sums + 255);
}

static void lora(int64_t a, int64_t b, int64_t c) {  // T, K, rank
    gemm_lora_t l = {};
    l.K = b, l.N = 1, l.adapters = 1, l.rank = c;
    l.lda = b, l.ldb = c;
    const LoraWorkspace w = lora_workspace(a, &l);
    CHECK(w.splits >= 1 && w.splits <= 4);
    CHECK(w.ldh >= c && w.ldh % 8 == 0);
    CHECK(w.parts % 256 == 0 && w.parts >= w.splits * a * w.ldh * 4);
    if (a > kLoraFew) {
        // three values of whole 16 tokens by 32 ranks, then a float for each token
        const int64_t tokens = (a + 15) / 16 * 16, ranks = (w.ldh + 31) / 32 * 32;
        CHECK(w.down % 16 == 0 && w.down >= w.parts + 3 * tokens * ranks * 2);
        CHECK(w.bytes >= w.down + 4 * a + 255);
    } else {
        CHECK(w.bytes >= w.parts + 255);
    }
}

int main() {
    const int64_t most = 0x7fffffff;
    const int64_t sizes[] = {1, 2, 7, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000, 2056, 4096,
                             8191, 16384, 65536, 1000000, most - 1, most};
    for (int64_t m : sizes)
        for (int64_t n : sizes)
            for (int64_t k : sizes) wgrad(m, n, k);
    const int64_t a = 0, b = 0, c = 0;
    CHECK(checkpoint_wgrad_workspace(0, 5, 5) == 0 && checkpoint_wgrad_workspace(5, 0, 5) == 0);
    CHECK(checkpoint_wgrad_workspace(-1, 5, 5) < 0 && checkpoint_wgrad_workspace(5, most + 1, 5) < 0);
    for (int64_t t : {1, 2, 15, 16, 17, 255, 256, 257, 300, 1000, 4096, 1 << 20})
        for (int64_t k : {1, 31, 511, 512, 513, 1024, 4096, 1 << 19})
            for (int64_t r : {1, 7, 8, 9, 16, 31, 32, 33, 64, 65, 200, 256}) lora(t, k, r);
    // the longest lines and the largest sizes are accepted, and addresses near the top refused
    // or accepted without overflow
    const int64_t line = (int64_t)1 << 40;
    CHECK(validate_checkpoint_pack(most, most, P(1 << 12), line, GEMM_BF16, P(1 << 13), line,
                                   reinterpret_cast<const uint8_t *>(P(1 << 14)), line) == GEMM_ERR_ALIASING);
    const uint64_t top = ~(uint64_t)0 - 4096;
    CHECK(validate_checkpoint_pack(1, 32, P(top), 32, GEMM_F32, P(1 << 12), 32,
                                   reinterpret_cast<const uint8_t *>(P(1 << 14)), 1) == GEMM_OK);
    CHECK(validate_checkpoint_wgrad(most, most, most, P(1 << 12), line, P(1 << 13), line,
                                    reinterpret_cast<const uint8_t *>(P(1 << 14)), line, nullptr, 0, P(1 << 15), line,
                                    GEMM_F16, GEMM_F32, nullptr, 0) == GEMM_ERR_ALIASING);
    CHECK(validate_moe_balance_dims(most, 1024, 32) == GEMM_OK && validate_moe_balance_dims(most + 1, 8, 2) != GEMM_OK);
    // sums of p and lse^2 in fp64, counts in int32, for each expert and one more
    CHECK(moe_balance_workspace(1024) >= kBalanceParts * 1025 * (8 + 4) + 255);
    printf("%d checks, %d failures\n", g_checked, g_fail);
    return g_fail != 0;
}
