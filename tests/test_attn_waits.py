"""The arithmetic of waiting in the tensor-core attention kernels (csrc/attn_waits.h), compiled for the host (CPU only).

The loaders' loops are written out again here over a model of barriers and copies, and made to give up at each of
their waits in turn."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "voxel_gemm_gb300", "csrc")


def run(tmp_path, source):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(source)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


LOADERS = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <utility>
#include "attn_waits.h"
using namespace vg;

// phases that copies (and the zeroing of a tail) complete on each barrier, in order; the last may be in flight
struct Model {
    std::map<std::pair<int, int>, int> phases;   // (barrier, slot) -> copies issued
    int waits = 0, stop;
    bool ok = true;
    explicit Model(int stop) : stop(stop) {}
    bool wait() { if (waits++ == stop) ok = false; return ok; }
    void copy(int bar, int slot) { ++phases[{bar, slot}]; }
    void seen(int bar, int slot, unsigned parity) {
        auto it = phases.find({bar, slot});
        if (it == phases.end() || it->second < 0) { printf("a wait for no copy\n"); exit(1); }
        if (((it->second - 1) & 1u) != parity) { printf("wrong phase of barrier %d slot %d\n", bar, slot); exit(1); }
        it->second = -1;
    }
    void all_seen() {
        for (auto& x : phases)
            if (x.second != -1) { printf("copy on barrier %d slot %d left in flight (stop %d)\n", x.first.first,
                                         x.first.second, stop); exit(1); }
    }
};
enum { Q, K, V, TAIL };
template <int S> void land(Model& m, const Copies<S>& c, int bar) {
    c.in_flight([&](uint32_t slot, uint32_t parity) { m.seen(bar, slot, parity); });
}

// forward: K and V of a tile by copies of their own; the sample's last V through the tail's barrier
template <int S> bool forward(int stop, int units, int tiles, bool cut) {
    Model m(stop);
    Copies<1> qs, tails;
    Copies<S> ks, vs;
    uint32_t at = 0;
    for (int u = 0; u < units && m.ok; ++u) {
        if (!m.wait()) break;
        m.copy(Q, 0);
        qs.issued();
        for (int e = 0; e < tiles; ++e, at = (at + 1) % S) {
            if (ks.slot() != at || vs.slot() != at || ks.pass() != (ks.n / S) % 2) { printf("wrong slot\\n"); exit(1); }
            if (!m.wait()) break;
            m.copy(K, at);
            ks.issued();
            if (!m.wait()) break;
            const bool last = cut && e + 1 == tiles;
            m.copy(last ? TAIL : V, last ? 0 : at);
            if (last) {
                tails.issued();
                m.wait();
                m.copy(V, at);                       // the arrival behind the zeroing
            }
            vs.issued();
        }
    }
    land(m, qs, Q), land(m, ks, K), land(m, vs, V), land(m, tails, TAIL);
    m.all_seen();
    return m.waits <= stop;
}
// backward: one barrier for the two tiles of a step
template <int S> bool backward(int stop, int units, int sets, int tiles, bool cut) {
    Model m(stop);
    Copies<1> qs, tails;
    Copies<S> steps;
    uint32_t at = 0;
    for (int u = 0; u < units && m.ok; ++u) {
        if (!m.wait()) break;
        m.copy(Q, 0);
        qs.issued();
        for (int h = 0; h < sets && m.ok; ++h)
            for (int e = 0; e < tiles; ++e, at = (at + 1) % S) {
                if (!m.wait()) break;
                const bool last = cut && e + 1 == tiles;
                m.copy(last ? TAIL : K, last ? 0 : at);
                if (last) {
                    tails.issued();
                    m.wait();
                    m.copy(K, at);
                }
                steps.issued();
            }
    }
    land(m, qs, Q), land(m, steps, K), land(m, tails, TAIL);
    m.all_seen();
    return m.waits <= stop;
}
int main() {
    for (int units = 0; units <= 4; ++units)
        for (int tiles = 1; tiles <= 7; ++tiles)
            for (int cut = 0; cut < 2; ++cut) {
                for (int stop = 0; !forward<2>(stop, units, tiles, cut); ++stop) {}
                for (int stop = 0; !forward<5>(stop, units, tiles, cut); ++stop) {}
                for (int sets = 1; sets <= 3; ++sets) {
                    for (int stop = 0; !backward<2>(stop, units, sets, tiles, cut); ++stop) {}
                    for (int stop = 0; !backward<4>(stop, units, sets, tiles, cut); ++stop) {}
                    for (int stop = 0; !backward<8>(stop, units, sets, tiles, cut); ++stop) {}
                }
            }
    printf("all seen\n");
}
"""


def test_no_copy_is_left_in_flight(tmp_path):
    """Wherever a loader gives up, the copies that it waits for at its end are all that can be in flight."""
    assert "all seen" in run(tmp_path, LOADERS)


LIMITS = r"""
#include <cstdio>
#include <cstdlib>
#include "attn_waits.h"
using namespace vg;

// The longest unit at `cycles` a step, against the limit of a wait for it.
void check(const char* what, int splits, int per, int64_t rows, int tile, int64_t sets, double steps) {
    const int64_t n = unit_steps(splits, per, rows, tile, sets);
    const double need = steps * 16 * 3000.0;       // 16 times what the slowest step takes
    if ((double)n < steps || (double)unit_wait_cycles(n) < need || unit_wait_cycles(n) < kWaitCycles) {
        printf("%s: %.3g steps take %.3g cycles, the wait gives up after %.3g\n", what, steps, need,
               (double)unit_wait_cycles(n));
        exit(1);
    }
}
int main() {
    const int64_t most = (int64_t(1) << 31) - 1;
    check("one tile", 1, 0, 5, 128, 1, 1);
    check("250 M packed rows against one tile of keys", 1, 0, 250000000, 64, 1, 250e6 / 64);
    check("as many rows as offsets allow, 8 head sets", 1, 0, most, 64, 8, 8.0 * most / 64);
    check("as many keys as offsets allow", 1, 0, most, 128, 1, most / 128.0);
    check("a part of them", 7, 2400000, most, 128, 1, 2400000);
    check("65,535 heads of as many rows", 1, 0, most, 64, 65535, 65535.0 * most / 64);
    if (unit_wait_cycles(INT64_MAX) < 0 || unit_wait_cycles(0) != kWaitCycles) return 1;
    printf("enough\n");
}
"""


def test_waits_for_units_last_as_long_as_the_longest(tmp_path):
    """A wait for a whole unit of work allows for the unit's steps, up to what 31-bit offsets and the heads can ask."""
    assert "enough" in run(tmp_path, LIMITS)
