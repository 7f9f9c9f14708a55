"""Build the HIP library in-tree with hipcc for gfx950.

``python -m block_max_qk_amd.build`` compiles the sources ``csrc/*.hip`` (one
object each, in parallel) and links them into
``block_max_qk_amd/libmsa_index_score.so``.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("msa_index_score.hip", "msa_attention.hip",
                                                   "msa_append.hip", "msa_tables.hip",
                                                   "msa_attention_forms_bf16.hip",
                                                   "msa_attention_forms_f16.hip")]
LIB = os.path.join(HERE, "libmsa_index_score.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def command(src: str, obj: str):
    return [HIPCC] + FLAGS + ["-I", os.path.join(ROOT, "include"),
                              "-I", os.path.join(HERE, "csrc"), "-c", src, "-o", obj]


def build(out: str = LIB, verbose: bool = False) -> str:
    tmp = out + ".tmp%d" % os.getpid()
    objs = ["%s.%d.o" % (tmp, i) for i in range(len(SOURCES))]
    cmds = [command(s, o) for s, o in zip(SOURCES, objs)]
    link = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        for cmd in cmds + [link]:
            print(" ".join(cmd), flush=True)
    try:
        running = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                   for c in cmds]
        said = [p.communicate()[0] for p in running]
        if all(p.returncode == 0 for p in running):
            r = subprocess.run(link, capture_output=True, text=True)
            if r.returncode == 0:
                os.replace(tmp, out)
                return out
            said.append(r.stdout + r.stderr)
        sys.stderr.write("".join(said))
        raise RuntimeError("hipcc failed building %s" % out)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)


if __name__ == "__main__":
    print(build(verbose=True))
