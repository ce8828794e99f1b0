"""The softmax warps' exchange of values (csrc/pair_exchange.h), compiled for the host: two threads go through the kernel's order of
waits and swaps, and each may leave at any of its waits.  Whatever the pair of places, both have to end, and
every value that a swap hands over has to be the other side's of the same step."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_moe_expert_router_gb300", "csrc")

HARNESS = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <mutex>
#include <thread>
#include "pair_exchange.h"

// A barrier of two arrivals that can be used again, as a named barrier of two warps; ends the program if a wait takes seconds.
struct State {
    std::mutex m;
    std::condition_variable cv;
    int arrived = 0;
    unsigned round = 0;
};
int fail_at[2];
struct Meet {
    State* s;
    void sync() {
        std::unique_lock<std::mutex> lock(s->m);
        const unsigned mine = s->round;
        if (++s->arrived == 2) {
            s->arrived = 0, ++s->round;
            s->cv.notify_all();
        } else if (!s->cv.wait_for(lock, std::chrono::seconds(3), [&] { return s->round != mine; })) {
            std::printf("a side waits for ever: they leave at their waits %d and %d\n", fail_at[0], fail_at[1]);
            std::_Exit(1);
        }
    }
    void arrive() {
        std::unique_lock<std::mutex> lock(s->m);
        if (++s->arrived == 2) {
            s->arrived = 0, ++s->round;
            s->cv.notify_all();
        }
    }
};

constexpr int kTiles = 3, kKeys = 3, kWaits = kTiles * (2 * kKeys + 1);

void side(int half, uint32_t* places, State* state, bool live, bool* wrong) {
    moe::PairExchange<Meet> other{places, 1, half, 0, {state}};
    int waits = 0, step = 0;
    bool ok = true;
    auto wait = [&] { return ok = waits++ != fail_at[half]; };
    auto exchange = [&] {
        const float nan = std::numeric_limits<float>::quiet_NaN();
        float x = step % 5 == 4 ? nan : 1000.f * half + step;  // (scores may be NaN)
        const bool there = other.swap(x);
        if (there && !(step % 5 == 4 ? x != x : x == 1000.f * (half ^ 1) + step)) *wrong = true;
        ++step;
        return ok = there;
    };
    for (int t = 0; ok && t < kTiles; ++t) {
        const bool has_rows = live || t != 1;  // a tile whose rows are none: waits without swaps
        for (int j = 0; j < kKeys; ++j) {
            if (!wait()) break;                                  // S
            if (has_rows && !exchange()) break;                  // the maxima
            if (j > 0 && j == t && !wait()) break;               // O before it is rescaled
        }
        if (!ok || !wait()) break;                               // the last P V
        if (has_rows && !exchange()) break;                      // the sums
    }
    if (!ok) other.leave();
    else exchange();
}

int main() {
    for (int live = 0; live < 2; ++live)
        for (fail_at[0] = -1; fail_at[0] < kWaits; ++fail_at[0])
            for (fail_at[1] = -1; fail_at[1] < kWaits; ++fail_at[1]) {
                uint32_t places[4] = {0, 0, 0, 0};
                State state;
                bool wrong[2] = {false, false};
                std::thread a(side, 0, places, &state, live == 1, wrong), b(side, 1, places, &state, live == 1, wrong + 1);
                a.join();
                b.join();
                if (wrong[0] || wrong[1]) {
                    std::printf("a value is not the other side's: they leave at their waits %d and %d\n", fail_at[0], fail_at[1]);
                    return 2;
                }
            }
    std::puts("all ended");
    return 0;
}
"""


def run(tmp_path, include):
    src, exe = tmp_path / "pair.cc", tmp_path / "pair"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", str(include), "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


def test_both_sides_end_wherever_either_leaves(tmp_path):
    r = run(tmp_path, CSRC)
    assert r.returncode == 0 and "all ended" in r.stdout, r.stdout


@pytest.mark.parametrize("line", ["meet.arrive();", "kLeftMark;\n        meet"], ids=["arrival", "mark"])
def test_the_check_finds_an_exchange_without_arrival_or_mark(tmp_path, line):
    """Without the arrival one side waits for ever; without the mark it goes on alone, to a later wait that never ends."""
    with open(os.path.join(CSRC, "pair_exchange.h")) as f:
        text = f.read()
    assert text.count(line) == 1
    (tmp_path / "inc").mkdir()
    (tmp_path / "inc" / "pair_exchange.h").write_text(text.replace(line, "" if line.startswith("meet") else "0;\n        meet"))
    r = run(tmp_path, tmp_path / "inc")
    assert r.returncode != 0, r.stdout
