"""Set-up that belongs to a device (a kernel's shared-memory limit, what fits on it) is done on every device of the
process, not once (CPU only: the helper with made-up devices, and the sources for statics that would hold one device's)."""
import glob
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_weight_only_quantize_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "per_device.cuh"
int main()
{
    static qerl::OncePerDevice once;
    int calls[3] = {0, 0, 0}, bad = 0;
    const auto ask = [&](int dev, int status) { return once(dev, [&] { ++calls[dev]; return status; }); };
    bad |= ask(0, 0) != 0 || ask(0, 7) != 0 || calls[0] != 1;                    // done: not asked again
    bad |= ask(1, 0) != 0 || calls[1] != 1;                                      // the second device sets up for itself
    bad |= ask(2, 5) != 5 || ask(2, 0) != 0 || ask(2, 5) != 0 || calls[2] != 2;  // a failure is tried again
    int other = 0;
    bad |= once(-1, [&] { ++other; return 0; }) != 0 || once(1 << 20, [&] { ++other; return 3; }) != 3 || other != 2;
    return bad;
}
"""


def test_every_device_is_set_up(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_static_holds_one_devices_answer():
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = open(path).read()
        assert not re.search(r"static\s+(?:const\s+)?\w+\s+\w+\s*=\s*cuda\w+\(", text), path
        assert "static std::atomic<int> fit[kMaxCluster" not in text
