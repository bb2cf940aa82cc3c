"""Programs for the host around the vocabulary operators' headers: what a kernel computes with
integers or fp32 alone can be looked at without a GPU."""
import os
import subprocess

import lm_head_vocab_gb300._lib as L

CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")


def run(tmp_path, source, *args):
    """Compile a C++ program that includes headers of csrc and return its output's lines."""
    src, exe = str(tmp_path / "program.cu"), str(tmp_path / "program")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run([L._nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2", "-I", CSRC,
                    "-o", exe, src], check=True)
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.splitlines()
