// The book of the expert products' tile counters, without a GPU: nobody holds a
// counter that another holds, what is given back is handed out again, and the
// book lives until its last holder lets go (run under the address sanitizer where
// there is one).
#include <stdio.h>

#include <thread>
#include <vector>

#include "tile_counters.h"

using ep::TileCounters;

#define CHECK(c)                                          \
    do {                                                  \
        if (!(c)) {                                       \
            printf("line %d: %s\n", __LINE__, #c);        \
            return 1;                                     \
        }                                                 \
    } while (0)

int main() {
    TileCounters *book = TileCounters::create();
    for (int i = 0; i < ep::kStreamCounters; ++i) CHECK(book->of_stream(1000 + 7 * i) == i);
    CHECK(book->of_stream(5) == -1 && book->of_stream(1007) == 1 && book->streams() == ep::kStreamCounters);

    std::vector<TileCounters::Captured *> held;
    std::vector<int> seen(ep::kStreamCounters + ep::kCapturedCounters, 0);
    for (int round = 0; round < 5; ++round) {   // as a program that captures its step again and again
        while (TileCounters::Captured *c = book->take()) {
            CHECK(c->index >= ep::kStreamCounters && c->index < (int)seen.size() && ++seen[c->index] == 1);
            held.push_back(c);
        }
        CHECK((int)held.size() == ep::kCapturedCounters && book->captured() == ep::kCapturedCounters);
        const size_t keep = round < 4 ? 100 : 8;
        while (held.size() > keep) {
            --seen[held.back()->index];
            TileCounters::give_back(held.back());
            held.pop_back();
        }
        CHECK(book->captured() == (int)keep);
    }
    // the handle goes first, the graphs' counters come back from several threads after it
    book->release();
    std::vector<std::thread> threads;
    for (TileCounters::Captured *c : held) threads.emplace_back([c] { TileCounters::give_back(c); });
    for (std::thread &t : threads) t.join();
    printf("ok\n");
    return 0;
}
