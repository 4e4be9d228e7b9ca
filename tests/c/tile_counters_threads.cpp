// The book of the counters under several host threads: those that meet new streams at the same time get one
// counter for each stream, the same in every thread, while captured calls come and go.
#include <stdio.h>

#include <atomic>
#include <thread>
#include <vector>

#include "tile_counters.h"

using ep::TileCounters;

int main() {
    constexpr int kThreads = 8, kIds = 300, kTurns = 40;
    for (int turn = 0; turn < kTurns; ++turn) {
        TileCounters *book = TileCounters::create();
        std::vector<std::vector<int>> got(kThreads, std::vector<int>(kIds, -2));
        std::atomic<int> ready{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < kThreads; ++t)
            threads.emplace_back([&, t] {
                ready.fetch_add(1);
                while (ready.load() < kThreads) {
                }
                for (int i = 0; i < kIds; ++i) {
                    const int id = t & 1 ? kIds - 1 - i : i;  // half of the threads from the other end
                    got[t][id] = book->of_stream(1000 + 7 * id);
                    if (i % 16 == t) {
                        TileCounters::Captured *c = book->take();
                        if (c != nullptr) TileCounters::give_back(c);
                    }
                }
            });
        for (std::thread &t : threads) t.join();
        std::vector<int> holder(ep::kStreamCounters, -1);
        for (int i = 0; i < kIds; ++i) {
            const int index = got[0][i];
            if (index < 0 || index >= ep::kStreamCounters || holder[index] != -1) {
                printf("stream %d: counter %d, held by %d\n", i, index, index >= 0 ? holder[index] : -1);
                return 1;
            }
            holder[index] = i;
            for (int t = 1; t < kThreads; ++t)
                if (got[t][i] != index) {
                    printf("stream %d: counters %d and %d\n", i, index, got[t][i]);
                    return 1;
                }
        }
        if (book->streams() != kIds || book->captured() != 0) {
            printf("%d streams, %d captured calls\n", book->streams(), book->captured());
            return 1;
        }
        book->release();
    }
    printf("ok\n");
    return 0;
}
