"""Host check of the order in which the gradient's issuing thread waits and issues (csrc/attention_order.h, the
same function the kernel runs) against a model of the barriers: rows that run as far ahead as their own waits let
them, or only when nothing else can go on, never bring it to a wait that cannot end, and no buffer is
overwritten before it has been read.  A parity waits for a phase that may already be two behind, as the hardware's does."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ulysses_sequence_attention_tf_gb300", "csrc")

HARNESS = r'''
#include <cstdio>
#include "attention_order.h"
using namespace tfu;

// A barrier: phases completed so far.  A wait for a parity ends when the phase in progress has the other one.
struct Bar { int done = 0; bool over(uint32_t parity) const { return (uint32_t(done) & 1u) != parity; } };

struct Model {
    int steps;
    bool eager;
    Bar s_full, dp_full, p, dx;
    int row = 0, at = 0;                       // the rows' step, and how far they are in it
    int s = -1, dp = -1, weighed = -1, updated = -1;  // what S and dP hold; the last P and dx that were taken
    long bad = 0;
    bool row_step() {                          // one action of the rows, if they can go on
        if (row >= steps) return false;
        const uint32_t parity = uint32_t(row) & 1u;
        if (at == 0) { if (!s_full.over(parity)) return false; bad += s != row; ++p.done; at = 1; return true; }
        if (!dp_full.over(parity)) return false;
        bad += dp != row; ++dx.done; at = 0; ++row;
        return true;
    }
    void run() { while (row_step()) {} }
    bool scores(int i) { bad += weighed != i - 1; s = i; ++s_full.done; if (eager) run(); return true; }
    bool gradients(int i) { bad += updated != i - 1; dp = i; ++dp_full.done; if (eager) run(); return true; }
    void weights(int i) { bad += row < i || (row == i && at == 0) || weighed != i - 1; weighed = i; if (eager) run(); }
    void update(int i) { bad += row <= i || updated != i - 1; updated = i; if (eager) run(); }
    bool wait(DqBarrier b, uint32_t parity) {
        Bar& bar = b == DqBarrier::kWeightsWritten ? p : dx;
        while (!bar.over(parity)) if (!row_step()) { ++bad; return false; }   // a wait that cannot end
        return true;
    }
};

// What the model has to find: dP(i + 1) issued before the wait for dx(i), on one barrier.
template <typename Pipe> bool ahead(int steps, Pipe& p) {
    if (!p.scores(0) || !p.gradients(0)) return false;
    for (int i = 0; i < steps; ++i) {
        if (!p.wait(DqBarrier::kWeightsWritten, i & 1u)) return false;
        p.weights(i);
        if (i + 1 < steps && (!p.scores(i + 1) || !p.gradients(i + 1))) return false;
        if (!p.wait(DqBarrier::kDxWritten, i & 1u)) return false;
        p.update(i);
    }
    return true;
}

int main() {
    long bad = 0, found = 0;
    for (int steps = 0; steps < 40; ++steps)
        for (int eager = 0; eager < 2; ++eager) {
            Model m{steps, eager != 0};
            const bool ok = dq_order(steps, m);
            m.run();
            bad += m.bad + !ok + (m.row != steps) + (m.updated != steps - 1) + (m.weighed != steps - 1);
            if (steps < 2) continue;
            Model n{steps, eager != 0};
            found += !ahead(steps, n) && eager;
        }
    std::printf("%ld %ld\n", bad, found);
    return bad != 0;
}
'''


def test_no_wait_of_the_gradient_expects_a_phase_that_has_passed(tmp_path):
    src = tmp_path / "order.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "order"
    subprocess.run(["g++", "-O2", "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    bad, found = r.stdout.split()
    assert r.returncode == 0 and bad == "0", r.stdout
    assert found == "38"  # the model does see it in an order that has the fault
