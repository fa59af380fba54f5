"""The launches that the model operators make for given sizes, recorded on the host without a GPU:
their C entry points and launch units, built host-only and linked with a stand-in for
hipLaunchKernel (tests/native/model_launch_check.cpp)."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

from dense_launches import CSRC, HERE, HIPCC, ROOT, record  # noqa: F401  (record: as there)

UNITS = [os.path.join(CSRC, u + ".hip") for u in
         ("qtcq_model", "launch_blocks", "launch_fp8", "launch_norm", "launch_distill")]


def build(folder, flags=()):
    """The recorder's path; flags: of its compilations and its link."""
    def one(src):
        obj = os.path.join(folder, os.path.basename(src) + ".o")
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC",
                        "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *flags, "-c", "-o", obj, src],
                       check=True, capture_output=True, text=True)
        return obj

    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(one, UNITS + [os.path.join(HERE, "native", "model_launch_check.cpp")]))
    exe = os.path.join(folder, "model_launch_check")
    # the host-only objects name GPU code that is not there
    subprocess.run(([HIPCC, *flags] if flags else ["g++"]) + ["-o", exe] + objs +
                   ["-Wl,--unresolved-symbols=ignore-in-object-files"],
                   check=True, capture_output=True, text=True)
    return exe
