"""Build libkda.so (gfx950) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkda.so")
SOURCES = ["kda_intra.hip", "kda_chain.hip", "kda_fused.hip", "kda_segment.hip", "kda_decode.hip", "kda_bwd.hip",
           "kda_api.hip", "kda_norm.hip", "kda_conv.hip", "kda_ssm.hip", "kda_ssm_bwd.hip", "kda_ssm_decode.hip",
           "kda_layer_api.hip", "kda_latent_fwd.hip", "kda_latent_bwd.hip", "kda_latent_decode.hip",
           "kda_latent_store.hip", "kda_latent_api.hip"]
HEADERS = [os.path.join(CSRC, h) for h in ("kda_common.h", "kda_intra_body.h", "kda_layer_args.h", "kda_ssm_common.h", "kda_checks.h",
                                                 "kda_latent_args.h", "kda_latent_common.h")] + [
    os.path.join(INCLUDE, h) for h in ("kda.h", "kda_layer.h", "kda_latent.h")]

# -packed-fp32-ops off: hipcc must not emit packed fp32 VALU instructions.
HIPCC_FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "hipcc"


# Per-source additions.  The state chain keeps its MFMA accumulators in
# ordinary VGPRs: the state update multiplies them by the decay every chunk, and
# accumulator-register copies around that multiply would sit on the serial path
# (the same in the state-space scan).
# The intra-chunk kernel is scheduled for instruction-level parallelism (it
# runs two workgroups per CU and spends much of each one's life on dependent
# chains): 1.2% faster than the default scheduler over 10 paired runs.
# The backward's per-chunk kernel runs one workgroup per CU (its LDS), so it may
# use the whole register file; in this form its overflow goes to accumulator
# registers rather than to scratch memory.
EXTRA_FLAGS = {"kda_ssm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "kda_ssm_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "kda_chain.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "kda_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "kda_fused.hip": ["-mllvm", "-amdgpu-sched-strategy=max-ilp"],
               "kda_intra.hip": ["-mllvm", "-amdgpu-sched-strategy=max-ilp"]}


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(verbose: bool = False) -> str:
    """Compile every HIP source into gated_delta_rule_110_amd/libkda.so (always rebuilds)."""
    tag = "%d" % os.getpid()
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(CSRC, src.replace(".hip", ".o%s" % tag))
        cmd = ([hipcc()] + [f for f in HIPCC_FLAGS if f != "-shared"] + EXTRA_FLAGS.get(src, [])
               + ["-c", "-I", INCLUDE, os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
        procs.append(_run(cmd, verbose))
    # the host pass warns that it does not know the packed-fp32 feature: harmless
    noise = "is not a recognized feature for this target"
    msgs, ok = [], True
    for p in procs:
        out = p.communicate()[0]
        msgs += [ln for ln in out.splitlines() if noise not in ln]
        ok = ok and p.returncode == 0
    tmp = LIB + ".tmp" + tag
    try:
        if ok:
            link = _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp], verbose)
            msgs += [ln for ln in link.communicate()[0].splitlines() if noise not in ln]
            ok = link.returncode == 0
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    if not ok:
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))
    os.replace(tmp, LIB)
    return LIB


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
