"""The distillation kernel's copies on devices of any number of SMs, on the CPU: csrc/distill_plan.h is
compiled as it is and every block's rows are gone through, with the slices, the copies that each row starts
(the phase its mbarriers then complete) and the phases that the waiting warps go by.  A wait for
another phase than the copy's would return before the copy is there, or never."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "layernorm_ln_fwd_gb300", "csrc")

SRC = r"""
#include <stdio.h>
#include <stdlib.h>
#include "distill_plan.h"
using namespace lnk;

// What a row's address leaves of it: vectors behind the first boundary of 16 bytes.
static int vectors(long long row, long long ld, int V, int es) {
    const int mis = (int)(row * ld * es % 16) / es, unit = 16 / es;
    const int head = (unit - mis) % unit;
    return (V - (head < V ? head : V)) / unit;
}

static long long uneven;  // uses of a slot with another number of copies than the use before

// `planted`: the mistake that a row arms only the copies that its own slice has.
static long long wrong(int rows, long long ld, int V, int es, int sms, int weights, bool planted) {
    const int nvec = V * es / 16;
    const DistillPlan plan = distill_plan(rows, nvec, sms, 4);
    if (plan.staged > kDsRoom || plan.chunk <= 0 || plan.copies > kDsChunks) {
        printf("no room: %d rows of %d\n", rows, V);
        exit(1);
    }
    const int at_once = plan.blocks > 1 ? sms / plan.blocks : plan.threads == 512 ? sms : 2 * sms;
    if (at_once < 1) return 0;
    const int stride = rows < at_once ? rows : at_once;
    long long bad = 0;
    for (int first = 0; first < stride; first += 1 + stride / 5)
        for (int rank = 0; rank < plan.blocks; ++rank) {
            unsigned armed[kDsSlots][kDsChunks] = {};
            int before[kDsSlots] = {-1, -1};
            SlotPhases phases;
            for (int row = first, slot = 0; row < rows; row += stride, slot ^= 1) {
                if (weights && (unsigned)row * 2654435761u >> 30 == 0) continue;  // weight 0: not read
                const int n = vectors(row, ld, V, es), per = (n + plan.blocks - 1) / plan.blocks;
                const int lo = n < rank * per ? n : rank * per, hi = n < lo + per ? n : lo + per;
                const int mid = hi < lo + plan.staged ? hi : lo + plan.staged;
                int copies = 0;
                for (int v = lo; v < mid; v += plan.chunk) ++copies;
                for (int i = 0; i < plan.copies; ++i)
                    if (i < copies || !planted) ++armed[slot][i];
                // The copy completes the phase that its arming began: the number of the armings before.
                for (int i = 0; i < copies; ++i)
                    bad += i >= plan.copies || phases.parity(slot) != ((armed[slot][i] - 1) & 1u);
                phases.used(slot);
                uneven += before[slot] >= 0 && before[slot] != copies;
                before[slot] = copies;
            }
        }
    return bad;
}

int main() {
    long long bad = 0, planted = 0, on152 = 0, calls = 0;
    const int slices[] = {1024, 1025, 2048, 2049, 3073, 4096, 4097, 6145, 6400};
    for (int sms = 2; sms <= 160; sms += sms < 60 ? 3 : 1)
        for (int es = 2; es <= 4; es += 2)
            for (int slice : slices)
                for (int blocks = 1; blocks <= 2; ++blocks)
                    for (int more = 0; more < 2; ++more)
                        for (int pad = 0; pad < 8; pad += 1 + 2 * more) {
                            const int V = slice * blocks * 16 / es + more;
                            for (int per = 1; per <= 5; per += 2) {
                                const int rows = per * 2 * sms - per;
                                for (int w = 0; w < 2; ++w, ++calls) {
                                    bad += wrong(rows, V + pad, V, es, sms, w, false);
                                    const long long p = wrong(rows, V + pad, V, es, sms, w, true);
                                    planted += p;
                                    if (sms == 152 && !w) on152 += p;
                                }
                            }
                        }
    printf("%lld %lld %lld %lld %lld\n", bad, planted, on152, uneven, calls);
    return 0;
}
"""


def test_every_wait_is_for_its_copy(tmp_path):
    cxx = shutil.which("c++") or shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "plan.cc"
    exe = tmp_path / "plan"
    src.write_text(SRC)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    bad, planted, on152, uneven, calls = map(int, run.stdout.split())
    assert bad == 0
    # The rows do differ in their copies, and arming those alone would be wrong.
    assert calls > 10000 and uneven > 1000 and planted > 1000, (calls, uneven, planted, on152)
