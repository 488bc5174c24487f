"""CPU checks of the limits of the expert operators' waits, compiled for the
host from the kernels' own source with a clock of the test's."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_block_scaled_route_b200", "csrc")

# A producer passes over `units` units of `cycles` cycles each, then arrives; every look at the barrier takes 1000 cycles.
MAIN = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#define __device__
#define __forceinline__ inline
#define __all_sync(mask, v) (v)
constexpr long long kWaitCycles = 2000000;
static long long now_ = 0, unit_cycles = 0, units = 0;
static bool stuck = false;
static volatile int moved_ = 0, abort_ = 0;
static long long clock64() { return now_; }
static bool mbar_try_wait(uint64_t*, uint32_t) {
  now_ += 1000;
  if (!stuck) moved_ = (int)(now_ / unit_cycles);
  return !stuck && now_ >= units * unit_cycles;
}
%s
static bool wait_of_the_fill_warp() {
  uint64_t fill[8] = {};
  uint32_t s = 0, uses = 0;
  volatile int *abort = &abort_, *moved = &moved_;
  (void)moved;
  bool ok = true;
  %s
  return ok;
}
static bool run(long long n, long long cycles, bool no_progress) {
  now_ = 0; moved_ = 0; abort_ = 0;
  units = n; unit_cycles = cycles; stuck = no_progress;
  return wait_of_the_fill_warp();
}
int main() {
  // any number of units ahead of the one waited for, each within the limit
  for (long long n : {1, 2, 7, 40})
    if (!run(n, kWaitCycles * 6 / 10, false) || abort_) return printf("gave up before unit %%lld\n", n), 1;
  // nothing moves: the wait ends, and soon after the limit
  if (run(1, 1, true) || !abort_ || now_ > 2 * kWaitCycles) return puts("no limit"), 1;
  // another role gave up: so does this one
  stuck = true; abort_ = 1; now_ = 0;
  if (wait_of_the_fill_warp() || now_ > kWaitCycles) return puts("abort not seen"), 1;
  puts("ok");
  return 0;
}
"""


def function(text, name):
    """Source of a function of the headers, from its qualifiers to the closing brace."""
    m = re.search(r"^__device__ __forceinline__ bool " + name + r"\(.*?^}\n", text, flags=re.S | re.M)
    return m.group(0) if m else ""


def test_weight_gradient_fill_waits_for_one_unit_at_a_time(tmp_path):
    """The warp that fills in a group's last rows passes over the units without such rows: its wait must not count the
    work of all of them against one limit."""
    with open(os.path.join(CSRC, "moe_ptx.cuh")) as f:
        ptx = f.read()
    with open(os.path.join(CSRC, "moe_grouped.cuh")) as f:
        grouped = f.read()
    with open(os.path.join(CSRC, "moe_wgrad.cu")) as f:
        call = re.search(r"ok = \w+\(&fill\[s\][^;]*;", f.read()).group(0)
    parts = [function(ptx, "mbar_wait")] + [function(grouped, n) for n in ("mbar_wait_warp", "mbar_wait_moving")]
    src, exe = tmp_path / "waits.cpp", tmp_path / "waits"
    src.write_text(MAIN % ("\n".join(parts), call))
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", str(exe), str(src)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
