"""Build tests/asan/train_asan: the C++ driver of the training step's entry
points, linked against libqlora's objects with their host code instrumented by
the address and undefined-behaviour sanitizers (device code as usual) and the
launchers replaced by the driver's.

    python tests/asan/build_train.py OUT_DIR
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
WRAPPED = ["_ZN5qlora16launch_gated_fwdERKNS_9GatedArgsEiRKNS_8CodebookEPKtPtS8_PfPvP12ihipStream_t",
           "_ZN5qlora16launch_gated_bwdERKNS_9GatedArgsERKNS_8CodebookEPKtS7_S7_PKfRKNS_10GatedGradsEPvP12ihipStream_t",
           "_ZN5qlora16launch_head_lossERKNS_12HeadLossArgsEPvP12ihipStream_t",
           "_ZN5qlora17launch_clip_gradsEiPKNS_10GradTensorEfPfPvP12ihipStream_t"]


def build(out_dir: str) -> str:
    os.makedirs(out_dir, exist_ok=True)
    hip, hip_host, cxx = B.sources()
    jobs = []
    for f in hip + hip_host:
        lang = [] if f.endswith(".hip") else ["-x", "hip"]
        jobs.append([B.HIPCC, *B.HIP_FLAGS, *B.FILE_FLAGS.get(f, []), *HOST_SAN, *lang, "-c", os.path.join(B.CSRC, f), "-o",
                     os.path.join(out_dir, f + ".o")])
    jobs.append([B.HIPCC, *B.HIP_FLAGS, *HOST_SAN, "-I", B.CSRC, "-x", "hip", "-c", os.path.join(HERE, "train_asan.cpp"),
                 "-o", os.path.join(out_dir, "train_asan.o")])
    for f in cxx:
        jobs.append(["g++", *B.CXX_FLAGS, "-c", os.path.join(B.CSRC, f), "-o", os.path.join(out_dir, f + ".o")])
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        list(ex.map(B._run, jobs))
    exe = os.path.join(out_dir, "train_asan")
    B._run([B.HIPCC, f"--offload-arch={B.ARCH}", "-fsanitize=address,undefined", "-fno-gpu-sanitize", "-o", exe,
            *[f"-Wl,--wrap={s}" for s in WRAPPED], *[j[-1] for j in jobs]])
    return exe


if __name__ == "__main__":
    print(build(sys.argv[1] if len(sys.argv) > 1 else os.path.join(HERE, "_build_train")))
