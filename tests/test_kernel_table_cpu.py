"""What the library remembers of a kernel is kept for the device it was set or
asked on, and nothing is kept where no device answers."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_13_gb300", "csrc")

PROGRAM = r"""
#include "kernel_table.h"
#include <cstdio>
#define CHECK(x) if (!(x)) { std::printf("failed: %s\n", #x); return 1; }
int main() {
    static pkv::KernelTable<int, 4> t;
    const int a = 0, b = 0;
    CHECK(!t.find(&a, 0));
    int *kept = t.add(&a, 0, 10);
    CHECK(kept && *kept == 10 && t.find(&a, 0) == kept);
    CHECK(!t.find(&a, 1) && !t.find(&b, 0));           // another device, another kernel
    CHECK(t.add(&a, 1, 11) && t.add(&b, 0, 20));
    CHECK(*t.find(&a, 0) == 10 && *t.find(&a, 1) == 11 && *t.find(&b, 0) == 20 && !t.find(&b, 1));
    CHECK(t.find(&a, 0) == kept);                      // entries stay where they are
    CHECK(!t.add(&b, -1, 30) && !t.find(&b, -1));      // no device: nothing is kept
    CHECK(t.add(&b, 1, 21) && !t.add(&a, 2, 12) && !t.find(&a, 2));   // full
    CHECK(*t.find(&b, 1) == 21);
    std::puts("ok");
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_entries_are_per_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_kernel_state_is_kept_by_function_alone():
    """Every static of the entry points that remembers a kernel is such a table; the others know no kernel."""
    with open(os.path.join(CSRC, "api.cu")) as f:
        statics = re.findall(r"^\s+static (?!const )([^=;(]*)[=;(]", f.read(), re.M)
    known = [s.strip() for s in statics]
    tables = [s for s in known if s.startswith("KernelTable<")]
    assert len(tables) == 4
    assert set(known) - set(tables) <= {"std::mutex mu", "std::once_flag once", "std::atomic<int> known[64]", "thread_local Fit4 f",
                                        "PFN_cuTensorMapEncodeTiled_v12000 fn"}
