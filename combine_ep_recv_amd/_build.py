"""Compile the HIP library in-tree for gfx950: combine_ep_recv_amd/libmoe_ep.so."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRC = os.path.join(CSRC, "moe_ep.hip")
SRCS = [SRC] + [os.path.join(CSRC, n) for n in ("moe_gate.hip", "moe_mx.hip")]
HDR = os.path.join(ROOT, "include", "moe_ep.h")
LIB = os.path.join(PKG, "libmoe_ep.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # keep the compiler from forming packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmds) -> str:
    """Run the commands side by side; their output without the host pass's note, or RuntimeError."""
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    texts = [p.communicate()[0] for p in procs]
    # the host pass does not know the packed-fp32 feature and says so; that is harmless
    noise = "is not a recognized feature for this target"
    outs = ["\n".join(l for l in t.splitlines() if noise not in l) for t in texts]
    for p, o in zip(procs, outs):
        if p.returncode != 0:
            raise RuntimeError("hipcc failed (%d):\n%s" % (p.returncode, o))
    return "\n".join(o for o in outs if o.strip())


def build() -> str:
    """Compile (always), one process per source, and return the path of the shared library."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp%d" % os.getpid()
    objs = ["%s.%d.o" % (tmp, i) for i in range(len(SRCS))]
    try:
        out = _run([[hipcc, *HIPCC_FLAGS, "-c", "-I", os.path.join(ROOT, "include"), "-o", o, s]
                    for s, o in zip(SRCS, objs)])
        out += _run([[hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]])
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    if out.strip():
        print(out)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
