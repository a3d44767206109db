"""How the decode step's workgroups wait for each other's flags (csrc/decode.hip), on the CPU.

The loop is compiled for the host as it stands, one lane of it, with a clock and flags of the test's own.
"""
import os
import re
import subprocess

import pytest

import mixture_experts_layer_02_amd.build as build

CLANG = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.HIPCC))), "llvm", "bin", "clang++")

HOST = r"""
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#define __HIP_MEMORY_SCOPE_AGENT 0
static uint64_t looks, up_after, jump_at, jump, every, numbers;
static uint64_t now() { return looks * every + (looks >= jump_at ? jump : 0); }
#define __builtin_amdgcn_s_memrealtime now
#define __builtin_amdgcn_s_sleep(n)
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __hip_atomic_load(p, order, scope) ((void)(p), uint32_t(looks >= up_after))
#define __hip_atomic_fetch_add(p, n, order, scope) ((void)(p), (uint32_t)numbers++)
static bool __all(bool all) { ++looks; return all; }
struct Params { uint32_t* sync; };
int main(int, char** a) {
  up_after = strtoull(a[1], 0, 0), jump_at = strtoull(a[2], 0, 0), jump = strtoull(a[3], 0, 0), every = strtoull(a[4], 0, 0);
  const int G = 256, lane = 0, SYNC_FLAGS = 128;
  numbers = strtoull(a[5], 0, 0);
  uint32_t sync[512] = {};
  Params p{sync};
  int nmore = 0;
  bool take = true;
LOOP
  printf("%d %llu\n", cmd, (unsigned long long)looks);
}
"""

SECOND = 100 * 10 ** 6  # of the 100 MHz clock
NEVER = 2 ** 62


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("wait")
    with open(os.path.join(build.CSRC, "decode.hip")) as fh:
        loop = re.search(r"\n( +int cmd = -1;\n.*?)\n +__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE", fh.read(), re.S).group(1)
    (tmp / "wait.cpp").write_text(HOST.replace("LOOP", loop))
    r = subprocess.run([CLANG, "-std=c++17", "-O2", "-w", str(tmp / "wait.cpp"), "-o", str(tmp / "wait")],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout

    def run(up_after, jump_at=NEVER, jump=0, every=150, numbers=256):
        out = subprocess.run([str(tmp / "wait")] + [str(v) for v in (up_after, jump_at, jump, every, numbers)],
                             stdout=subprocess.PIPE, text=True, timeout=60, check=True).stdout
        return tuple(int(v) for v in out.split())
    return run


def test_goes_on_when_all_flags_are_up(wait):
    assert wait(up_after=0)[0] == -1
    assert wait(up_after=5) == (-1, 6)


def test_takes_a_number_that_nobody_has_started_on(wait):
    cmd, looks = wait(up_after=1000, numbers=200)
    assert cmd == 200 and looks < 30  # (after 20 us)


@pytest.mark.parametrize("seconds", [1, 11, 3600])
def test_a_queue_taken_off_the_gpu_does_not_end_the_wait(wait, seconds):
    """The clock runs on while the waves do not: hours between two looks are no reason to give up."""
    assert wait(up_after=40, jump_at=20, jump=seconds * SECOND) == (-1, 41)


def test_a_wait_without_an_end_is_given_up(wait):
    """Flags that another call cleared never come: the kernel ends, after looks of at least 1 us that last some seconds."""
    cmd, looks = wait(up_after=NEVER)
    assert cmd == -2 and 5 * 10 ** 6 <= looks <= 20 * 10 ** 6
