"""Build libar.so (the C-ABI library with the gfx950 kernels) in-tree with hipcc.

Every source is compiled to an object of its own, several at a time (the
kernel families live in separate translation units), and the objects are
linked into one shared library."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libar.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = ["ar_kernels_ring_simple.hip", "ar_kernels_ring_ll.hip", "ar_kernels_ring_ll128.hip", "ar_kernels_ring_batch.hip",
           "ar_kernels_ring_rs.hip", "ar_kernels_ring_ag.hip", "ar_kernels_tree.hip", "ar_kernels_tree_batch.hip",
           "ar_kernels.hip", "ar_noalloc.hip", "ar_layernorm.hip", "ar_gradnorm.hip", "ar_dropout.hip",
           "ar_logprob.hip", "ar_policy.hip",
           "ar_comm.cpp", "ar_tune.cpp", "ar_group.cpp", "ar_api.cpp"]
ARCH = os.environ.get("AR_OFFLOAD_ARCH", "gfx950")
ROCM_LIB = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "lib")
FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
         # every add is one IEEE add; binary32 subnormals are kept
         "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
         # no packed-FP32 instructions: each float add is one lane's own add
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _jobs():
    return max(1, min(len(SOURCES), os.cpu_count() or 1, 16))


TUNE_TABLE = os.path.join(CSRC, "ar_tune_table.txt")


def parse_tune_table(path):
    """(rows, models) of a tuner table file: rows are (ranks, bytes, six
    microsecond times or None), models map (algo, proto) to the four model
    constants.  The library reads the same format at run time (AR_TUNE_FILE)."""
    rows, models = [], {}
    for line in open(path):
        line = line.split("#", 1)[0].split()
        if not line:
            continue
        if line[0] == "model":
            models[(line[1], line[2])] = [float(x) for x in line[3:7]]
            continue
        rows.append((int(line[0]), int(line[1]), [None if x == "-" else float(x) for x in line[2:8]]))
    return rows, models


def write_tune_table_inc(out):
    """The compiled tuner table and model constants, from ar_tune_table.txt."""
    rows, models = parse_tune_table(TUNE_TABLE)
    lines = ["// Generated by build.py from ar_tune_table.txt; do not edit.",
             "static const ar::TuneRow kCompiledTuneRows[] = {"]
    for n, b, ts in rows:
        lines.append("    {%d, %dull, {%s}}," % (n, b, ", ".join("-1.0f" if t is None else "%.3ff" % t for t in ts)))
    lines.append("};")
    for algo in ("ring", "tree"):
        lines.append("static const arTuneModel_t kCompiled%sModels[3] = {" % algo.capitalize())
        for proto in ("ll", "ll128", "simple"):
            m = models[(algo, proto)]
            lines.append("    {%.4ff, %.4ff, %.4ff, %.4ff},  // %s" % (m[0], m[1], m[2], m[3], proto))
        lines.append("};")
    text = "\n".join(lines) + "\n"
    if not os.path.exists(out) or open(out).read() != text:
        with open(out, "w") as f:
            f.write(text)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    write_tune_table_inc(os.path.join(OBJ, "ar_tune_table.inc"))
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", OBJ]

    def compile_one(src):
        obj = os.path.join(OBJ, src + ".o")
        cmd = ["hipcc"] + FLAGS + inc + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(max_workers=_jobs()) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    # ROCTx ranges on the API entry points (rocprofv3 --marker-trace)
    cmd = ["hipcc", "--offload-arch=" + ARCH, "-shared", "-fPIC"] + objs + [
        "-L" + ROCM_LIB, "-Wl,-rpath," + ROCM_LIB, "-lrocprofiler-sdk-roctx", "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    build_torch_calls(verbose)
    build_probe(verbose)
    return LIB


TORCH_CALLS = os.path.join(HERE, "_ar_torch.so")


def built_for() -> str:
    """The Python and torch the extension module belongs to: it uses their C++ layouts."""
    import sys
    import torch
    return "python %d.%d, torch %s" % (sys.version_info[0], sys.version_info[1], torch.__version__)


def build_torch_calls(verbose: bool = False) -> str:
    """The extension module that reads torch tensors for binding.py (host code only)."""
    import sysconfig
    import torch
    t = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), '-DAR_BUILT_FOR="%s"' % built_for(),
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(rocm, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(CSRC, "ar_torch.cpp"), "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip",
           "-L" + ROCM_LIB, "-lamdhip64", "-Wl,-rpath," + ROCM_LIB, "-o", TORCH_CALLS + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(TORCH_CALLS + ".tmp", TORCH_CALLS)
    return TORCH_CALLS


PROBE_LIB = os.path.join(HERE, "libstream_ceiling.so")


def build_probe(verbose: bool = False) -> str:
    """The streaming-ceiling probe bench.py reports beside the HBM peak."""
    cmd = ["hipcc", "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           os.path.join(CSRC, "probes", "stream_ceiling.hip"), "-o", PROBE_LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(PROBE_LIB + ".tmp", PROBE_LIB)
    return PROBE_LIB


if __name__ == "__main__":
    print(build(verbose=True))
