// The shares that the attention cuts its steps into (q8_kv4_shares.h),
// compiled for the host: they cover the room in order, none is empty where
// the layout needs every one, every position finds its share, and a search
// ends whatever it looks for.  The exit status is the number of the check that failed.
#include <cstdint>
#include <random>

#include "q8_kv4_shares.h"

int main() {
    std::mt19937_64 rng(1);
    for (int on_cu = 1; on_cu <= 3; ++on_cu)
        for (int n : {1, 2, 3, 5, 8, 31, 32, 96, 102, 153, 255, 256, 391, 511, 512, 767, 768})
            for (int trial = 0; trial < 200; ++trial) {
                const bool even = trial % 2 == 0;
                const int64_t least = even ? 1 : (int64_t)q8::kMinSteps * n + 1;
                const int64_t most = even ? (int64_t)q8::kMinSteps * n
                                          : trial % 3 == 0 ? least + 100 : trial % 3 == 1 ? least * 50 : int64_t(1) << 43;
                const int64_t room = least + (int64_t)(rng() % (uint64_t)(most - least + 1));
                const q8::Shares s(room, n, even, on_cu);
                if (s.start(0) != 0 || s.start(n) != room || s.start(n + 1) != room) return 1;
                for (int i = 0; i < n; ++i) {
                    const int64_t a = s.start(i), b = s.start(i + 1);
                    if (b < a || (!even && b == a)) return 2;
                    if (b > a && (s.at(a) != i || s.at(b - 1) != i)) return 3;
                    if (b > a && s.at(a + (int64_t)(rng() % (uint64_t)(b - a))) != i) return 4;
                }
                for (int64_t past : {room, room + 1, room + 12345, int64_t(1) << 44})
                    if (s.at(past) != n - 1) return 5;
            }
    return 0;
}
