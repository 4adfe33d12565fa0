"""The rounds that the warps of a group make together (csrc/rounds.cuh), compiled for the host:
members that give up, at any round and apart from one another, leave no other one waiting at the
group's barrier, which has no time limit on the device."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sliding_window_anchor_b200", "csrc")

SOURCE = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>
#include "rounds.cuh"

constexpr int kMembers = 8;

// A barrier of all members; one that waits too long is counted and lets everybody go.
struct Barrier {
  std::mutex mu;
  std::condition_variable cv;
  int waiting = 0, turn = 0, stuck = 0;
  void sync(int ms) {
    std::unique_lock<std::mutex> lock(mu);
    const int mine = turn;
    if (++waiting == kMembers) {
      waiting = 0, ++turn;
      cv.notify_all();
      return;
    }
    if (!cv.wait_for(lock, std::chrono::milliseconds(ms),
                     [&] { return turn != mine || stuck; }))
      ++stuck;
    if (stuck) cv.notify_all();
  }
};

// Rounds as the kernel makes them: one meeting, then what may give up.  `rest`: a member
// that gives up meets the others in the rounds that it leaves out.
template <class Meet, class Round>
void make_rounds(bool rest, int n, Meet&& meet, Round&& round) {
  int c = 0;
  for (; c <= n; ++c) {
    meet();
    if (!round(c)) break;
  }
  if (rest) er::meet_rest(c, n, meet);
}

// Members of the mask give up in round `at`, every second one of them one round later.
bool ends(bool rest, int n, unsigned mask, int at, int ms, long* done) {
  Barrier bar;
  std::vector<std::thread> members;
  std::vector<int> work(kMembers, 0), late(kMembers, 0);
  for (int i = 0; i < kMembers; ++i)
    members.emplace_back([&, i] {
      const int last = (mask >> i & 1) ? at + (i & 1) : n + 1;
      make_rounds(rest, n, [&] { bar.sync(ms); },
                  [&](int c) {
                    ++work[i];
                    if (c > last) late[i] = 1;
                    return c < last;
                  });
    });
  for (auto& m : members) m.join();
  for (int i = 0; i < kMembers; ++i) {
    *done += work[i];
    const int last = (mask >> i & 1) ? at + (i & 1) : n + 1;
    if (!bar.stuck && (late[i] || work[i] != (last < n ? last : n) + 1)) return false;
  }
  return !bar.stuck;
}

int main() {
  long done = 0;
  for (int n : {1, 2, 5})
    for (int at = 0; at <= n; ++at)
      for (unsigned mask : {0u, 1u, 2u, 0x80u, 0x0Fu, 0x33u, 0x7Fu, 0xFFu})
        if (!ends(true, n, mask, at, 20000, &done)) {
          std::printf("stuck or wrong: n %d mask %x at %d\n", n, mask, at);
          return 1;
        }
  // the harness sees members that are left alone
  if (ends(false, 3, 1u, 1, 200, &done)) {
    std::printf("not seen\n");
    return 1;
  }
  std::printf("ok %ld\n", done);
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("rounds")
    src, exe = d / "rounds.cpp", d / "rounds"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-o", str(exe),
                           str(src)])
    return str(exe)


def test_no_member_is_left_at_the_barrier(program):
    out = subprocess.run([program], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    assert out.stdout.startswith("ok")
