"""The shared-memory limit of a kernel under two host threads (C++, no GPU): it ends at the
larger request and is never lowered."""
import os
import subprocess

import weight_streaming_warp_gb300 as wsw

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <future>
#include <thread>

#include "smem_grant.h"

int main() {
    using namespace std::chrono_literals;
    static int kernel;
    wsw::SmemGrants grants;
    std::atomic<int> limit{0}, sets{0};  // the limit as CUDA would hold it
    std::promise<void> inside, go;
    std::thread small([&] {
        grants.ensure(&kernel, 0, 20, [&](int n) {
            inside.set_value();
            go.get_future().wait();
            limit = n;
            ++sets;
            return 0;
        });
    });
    inside.get_future().wait();  // the smaller request is about to set its limit
    std::promise<void> done;
    std::thread large([&] {
        grants.ensure(&kernel, 0, 1000, [&](int n) { limit = n; ++sets; return 0; });
        done.set_value();
    });
    done.get_future().wait_for(300ms);  // it may have to wait for the first
    go.set_value();
    small.join();
    large.join();
    if (limit != 1000) return std::printf("ends at %d\n", limit.load()), 1;
    auto fail = [&](int) { ++sets; return 7; };
    const int before = sets;
    if (grants.ensure(&kernel, 0, 20, fail) || grants.ensure(&kernel, 0, 1000, fail) || sets != before)
        return std::puts("a granted size is set again"), 1;
    if (grants.ensure(&kernel, 0, 2000, fail) != 7 || grants.ensure(&kernel, 1, 20, fail) != 7 ||
        grants.ensure(&sets, 0, 20, fail) != 7)
        return std::puts("an error is lost"), 1;
    if (grants.ensure(&kernel, 0, 2000, [&](int n) { limit = n; return 0; }) || limit != 2000)
        return std::puts("a refused size counts as granted"), 1;
    return 0;
}
"""


def test_two_threads_end_at_the_larger_limit(tmp_path):
    src = tmp_path / "grants.cpp"
    src.write_text(PROGRAM)
    include = os.path.join(os.path.dirname(wsw.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", include, str(src), "-o", str(tmp_path / "grants")],
                   check=True)
    r = subprocess.run([str(tmp_path / "grants")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
