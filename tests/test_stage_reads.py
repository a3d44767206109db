"""Where the streaming kernels' reads of an LDS stage end (csrc/stream.h), on the CPU.

A ring's stages are sized for the activation rows that a call has, and the last stage of
the last wave ends where LDS ends.  Stage::read is compiled for the host here and
reads stages that end at a page without access, for every form that decode.hip and
i4.hip launch and every number of rows.
"""
import itertools
import os
import re
import subprocess

import mixture_experts_layer_02_amd.build as build

CLANG = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.HIPCC))), "llvm", "bin", "clang++")

# What stream.h takes from the device's headers; copies and products do nothing.
STUB = r"""
#pragma once
#include <stdint.h>
#include <type_traits>
#define __device__
#define __host__
#define __forceinline__ inline
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_s_waitcnt(x)
#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16 product
namespace moe {
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
template <typename T> constexpr T min(T a, T b) { return a < b ? a : b; }
template <typename A, typename C> C product(A, A, C c, int, int, int) { return c; }
inline uint32_t __umul24(uint32_t a, uint32_t b) { return a * b; }
namespace dma {
typedef int i32x4 __attribute__((ext_vector_type(4)));
inline i32x4 make_rsrc(const void*, uint64_t) { return i32x4{}; }
inline void dma16(i32x4, uint32_t, uint32_t, uint32_t) {}
inline void touch4u(i32x4, uint32_t, uint32_t, uint32_t) {}
template <int N> inline void wait_vm() {}
}
}
"""

MAIN = r"""
#include "stream.h"
#include <setjmp.h>
#include <signal.h>
#include <stdio.h>
#include <string.h>
#include <sys/mman.h>
using namespace moe::stream;
static sigjmp_buf back;
static void fault(int) { siglongjmp(back, 1); }
static uint8_t* top;  // the end of what may be read
template <int GRP, int R, int SUB, bool DUAL, int RB> void check(const char* name) {
  using ST = Stage<GRP, R, SUB, DUAL, RB>;
  for (int rows = 1; rows <= RB; ++rows) {
    const uint8_t* slot = top - ST::bytes(rows);
    int bad = 0;
    for (int lane = 0; lane < 64; ++lane) {
      if (sigsetjmp(back, 1)) { ++bad; continue; }
      ST s;
      s.read(slot, lane, ST::column(lane, rows));
      asm volatile("" : : "r"(&s) : "memory");
      // a lane whose column exists reads that column
      if ((lane & 15) < rows && ST::column(lane, rows) != (lane & 15)) printf("%s: lane %d, %d rows: another column\n", name, lane, rows);
    }
    if (bad) printf("%s: %d rows: %d lanes read past the stage\n", name, rows, bad);
  }
}
int main() {
  const size_t n = 1 << 20;
  uint8_t* p = (uint8_t*)mmap(nullptr, n + 65536, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  if (p == MAP_FAILED || mprotect(p + n, 65536, PROT_NONE)) return 2;
  top = p + n;
  struct sigaction a = {};
  a.sa_handler = fault;
  sigaction(SIGSEGV, &a, nullptr);
  sigaction(SIGBUS, &a, nullptr);
FORMS
  puts("done");
}
"""


def _forms():
    """(GRP, R, SUB, DUAL, RB) of every stage that decode.hip and i4.hip use."""
    with open(os.path.join(build.CSRC, "decode.hip")) as fh:
        runs = re.findall(r"run<([^>]+)>\(p, grid, s\)", fh.read())
    assert len(runs) >= 14
    out = set()
    for args in runs:
        grp, _, rb, r1, r2, sub2, _ = (a.strip() for a in args.split(","))
        for g in ((0,) if grp == "0" else (32, 64, 128)):
            out |= {(g, int(r1), 1, 1, int(rb)), (g, int(r2), int(sub2), 0, int(rb))}
    with open(os.path.join(build.CSRC, "i4.hip")) as fh:
        linear = re.findall(r"run_linear<GRP, (\d+), (\d+), OUT>\(p, s\)", fh.read())
    assert len(linear) >= 5
    return sorted(out | {(g, int(r), 1, 0, int(rb)) for g, (rb, r) in itertools.product((32, 64, 128), linear)})


def test_reads_stay_within_a_stage(tmp_path):
    with open(os.path.join(build.CSRC, "stream.h")) as fh:
        text = fh.read()
    # (device assembly: memory clobbers, waits and the copies' instructions)
    text = re.sub(r"\basm\s*(?:volatile)?\s*\((?:[^()\"]|\"[^\"]*\"|\([^()]*\))*\)\s*;", ";", text)
    (tmp_path / "stream.h").write_text(text)
    (tmp_path / "gemm_dma.h").write_text(STUB)
    calls = "\n".join(f'  check<{g}, {r}, {sub}, {"true" if dual else "false"}, {rb}>("{g}/{r}/{sub}/{dual}/{rb}");'
                      for g, r, sub, dual, rb in _forms())
    (tmp_path / "main.cpp").write_text(MAIN.replace("FORMS", calls))
    r = subprocess.run([CLANG, "-std=c++17", "-O1", "-w", str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([str(tmp_path / "main")], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert (r.returncode, r.stdout) == (0, "done\n"), r.stdout
