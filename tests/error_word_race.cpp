// Threads that ask for an error word at the same moment, many times over: of those that ask after it was
// latched once, exactly one is to be told. Prints how many rounds there were, told nobody, and told several.
#include <barrier>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include "error_word.h"

int main(int argc, char** argv) {
  const int rounds = std::atoi(argv[1]), threads = std::atoi(argv[2]);
  unsigned memory = 0;
  fh::ErrorWord word;
  if (word.take()) return 1;  // not allocated: nothing to tell
  word.host.store(&memory);
  std::atomic<int> told{0};
  int none = 0, several = 0;
  std::barrier begin(threads + 1), end(threads + 1);
  std::vector<std::thread> asking;
  for (int t = 0; t < threads; ++t)
    asking.emplace_back([&] {
      for (int r = 0; r < rounds; ++r) {
        begin.arrive_and_wait();
        if (word.take() == 1u) told.fetch_add(1);
        end.arrive_and_wait();
      }
    });
  for (int r = 0; r < rounds; ++r) {
    told = 0;
    __atomic_fetch_or(&memory, 1u, __ATOMIC_RELEASE);
    begin.arrive_and_wait();
    end.arrive_and_wait();
    none += told == 0;
    several += told > 1;
  }
  for (auto& t : asking) t.join();
  std::printf("%d %d %d\n", rounds, none, several);
  return memory != 0;
}
