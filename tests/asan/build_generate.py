"""Build tests/asan/generate_asan: the C++ driver of the attention side's entry
points, linked against libqlora's objects with their host code instrumented by
the address and undefined-behaviour sanitizers (device code as usual) and the
launchers replaced by the driver's.

    python tests/asan/build_generate.py OUT_DIR
"""

from __future__ import annotations

import concurrent.futures
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
sys.path.insert(0, ROOT)

from bit_nf4_quantized_21_amd import build as B  # noqa: E402

SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize=vptr,function", "-fno-sanitize-recover=all",
       "-fno-omit-frame-pointer", "-g"]
HOST_SAN = [a for s in SAN for a in ("-Xarch_host", s)]
WRAPPED = ["_ZN5qlora13launch_attendERKNS_13AttendProblemEPKfPvP12ihipStream_t",
           "_ZN5qlora11launch_ropeEliRKNS_9RopeTableEbRKNS_9HeadsViewES5_S5_S5_P12ihipStream_t",
           "_ZN5qlora17launch_rope_tableERKNS_13RopeTableArgsEPfP12ihipStream_t",
           "_ZN5qlora15launch_kv_writeERKNS_6KVPoolElRKNS_9HeadsViewES5_PKlRKNS_9RopeTableERKNS_9MidpointsEP12ihipStream_t",
           "_ZN5qlora14launch_kv_readERKNS_6KVPoolElPKlPtS5_PKfP12ihipStream_t"]


def build(out_dir: str) -> str:
    os.makedirs(out_dir, exist_ok=True)
    hip, hip_host, cxx = B.sources()
    jobs = []
    for f in hip + hip_host:
        lang = [] if f.endswith(".hip") else ["-x", "hip"]
        jobs.append([B.HIPCC, *B.HIP_FLAGS, *B.FILE_FLAGS.get(f, []), *HOST_SAN, *lang, "-c", os.path.join(B.CSRC, f), "-o",
                     os.path.join(out_dir, f + ".o")])
    jobs.append([B.HIPCC, *B.HIP_FLAGS, *HOST_SAN, "-I", B.CSRC, "-x", "hip", "-c", os.path.join(HERE, "generate_asan.cpp"),
                 "-o", os.path.join(out_dir, "generate_asan.o")])
    for f in cxx:
        jobs.append(["g++", *B.CXX_FLAGS, "-c", os.path.join(B.CSRC, f), "-o", os.path.join(out_dir, f + ".o")])
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        list(ex.map(B._run, jobs))
    exe = os.path.join(out_dir, "generate_asan")
    B._run([B.HIPCC, f"--offload-arch={B.ARCH}", "-fsanitize=address,undefined", "-fno-gpu-sanitize", "-o", exe,
            *[f"-Wl,--wrap={s}" for s in WRAPPED], *[j[-1] for j in jobs]])
    return exe


if __name__ == "__main__":
    print(build(sys.argv[1] if len(sys.argv) > 1 else os.path.join(HERE, "_build_generate")))
