"""The launches that the dense operators make for given sizes, recorded on the host without a
GPU: their C entry points and launch units, built host-only and linked with a stand-in for
hipLaunchKernel (tests/native/dense_launch_check.cpp)."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "trellis_coded_weight_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
UNITS = [os.path.join(CSRC, u + ".hip") for u in
         ("qtcq_dense", "launch_rows", "launch_int8", "launch_gated", "launch_gated_vjp")]


def build(folder):
    """The recorder's path."""
    def one(src):
        obj = os.path.join(folder, os.path.basename(src) + ".o")
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC",
                        "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c", "-o", obj, src],
                       check=True, capture_output=True, text=True)
        return obj

    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(one, UNITS + [os.path.join(HERE, "native", "dense_launch_check.cpp")]))
    exe = os.path.join(folder, "dense_launch_check")
    # the host-only objects name GPU code that is not there
    subprocess.run(["g++", "-o", exe] + objs + ["-Wl,--unresolved-symbols=ignore-in-object-files"],
                   check=True, capture_output=True, text=True)
    return exe


def record(exe, calls):
    """For each call (a line of the recorder's input): (status, [words of a launch])."""
    r = subprocess.run([exe], input="\n".join(calls) + "\n", capture_output=True, text=True, check=True, timeout=300)
    out, launches = [], []
    for line in r.stdout.splitlines():
        words = line.split()
        if words[0] == "=":
            out.append((int(words[1]), launches))
            launches = []
        else:
            launches.append(words)
    assert len(out) == len(calls)
    return out
