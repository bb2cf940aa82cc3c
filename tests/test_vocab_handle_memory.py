"""The handle's memory on the host, over a runtime whose cudaMemset returns before it is done, as the
real one's does: a stream that does not wait for the legacy one must find the counters at zero."""
import os
import shutil
import subprocess

import pytest

import lm_head_vocab_gb300._lib as L

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")
CUDA = "/usr/local/cuda"


def run(tmp_path, unit, body):
    """Compile one source file of the library, link it with the stand-in runtime, run `body`."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    main, obj, lib, exe = (str(tmp_path / n) for n in ("main.cpp", "unit.o", "libunit.so", "main"))
    with open(main, "w") as f:
        f.write('#include <cstdio>\n#include "lmloss.h"\n#include <cuda_runtime_api.h>\nint unfinished_fills();\nint main()\n{\n' + body + "    return 0;\n}\n")
    subprocess.run([L._nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O1", "-Xcompiler", "-fPIC",
                    "-c", "-o", obj, os.path.join(CSRC, unit)], check=True)
    cxx = [cxx, "-std=c++17", "-fPIC", "-I", os.path.join(HERE, "..", "include"), "-I", os.path.join(CUDA, "include")]
    # what `body` does not reach stays unresolved
    subprocess.run([*cxx, "-shared", "-Wl,-z,lazy", "-o", lib, os.path.join(HERE, "vocab_fake_runtime.cpp"), obj], check=True)
    subprocess.run([*cxx, "-Wl,-z,lazy", "-Wl,--allow-shlib-undefined", "-o", exe, main, lib, "-Wl,-rpath," + str(tmp_path),
                    "-lpthread"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_counters_are_zero_when_create_returns(tmp_path):
    run(tmp_path, "vocab_handle.cu", """
    lmloss_vocab_handle h;
    if (lmloss_vocab_create(&h, 0, 1 << 20) != LMLOSS_OK) return 1;
    if (unfinished_fills() != 0) return std::printf("create returned before its memory was zero\\n"), 2;
    if (lmloss_vocab_destroy(h) != LMLOSS_OK) return 3;
""")


def test_the_error_word_is_clear_when_it_has_been_read(tmp_path):
    run(tmp_path, "vocab_handle.cu", """
    lmloss_vocab_handle h;
    if (lmloss_vocab_create(&h, 0, 0) != LMLOSS_OK || lmloss_vocab_get_device_error(h) != LMLOSS_OK) return 1;
    if (unfinished_fills() != 0) return std::printf("the next call's error may still be cleared\\n"), 2;
    if (lmloss_vocab_destroy(h) != LMLOSS_OK) return 3;
""")


def test_the_loss_handle_keeps_to_the_same(tmp_path):
    run(tmp_path, "lmloss.cu", """
    lmloss_handle h;
    if (lmloss_create(&h, 0, 1024, 4) != LMLOSS_OK) return 1;
    if (unfinished_fills() != 0) return std::printf("create returned before its memory was zero\\n"), 2;
    if (lmloss_get_device_error(h) != LMLOSS_OK) return 3;
    if (unfinished_fills() != 0) return std::printf("the next call's error may still be cleared\\n"), 4;
    if (lmloss_destroy(h) != LMLOSS_OK) return 5;
""")


@pytest.mark.parametrize("unit,handle,create", [("vocab_handle.cu", "lmloss_vocab_handle", "lmloss_vocab_create(&h, 9, 0)"),
                                                ("lmloss.cu", "lmloss_handle", "lmloss_create(&h, 9, 16, 1)")])
def test_a_device_that_is_not_there_leaves_no_error_behind(tmp_path, unit, handle, create):
    # the next call's check of its launch would find it
    run(tmp_path, unit, f"""
    {handle} h;
    if ({create} != LMLOSS_ERR_CUDA) return 1;
    if (cudaGetLastError() != cudaSuccess) return std::printf("an error is left for the next call\\n"), 2;
""")


def test_the_fixed_workspace_is_not_cleared_under_its_first_call():
    # it is zero when the module loads; its set-up runs inside the first call
    text = open(os.path.join(CSRC, "lmloss.cu")).read()
    setup = text[text.index("lmloss_status noalloc_setup"):text.index('extern "C" lmloss_status lmloss_forward_backward_noalloc')]
    assert "static __device__ __align__(256) unsigned char g_noalloc_scratch" in text and "Memset" not in setup


@pytest.mark.gpu
def test_calls_after_a_handle_on_a_device_that_is_not_there():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    ops = VocabOps(0, max_tokens=0, max_rows=0)
    w, ids = torch.randn(9, 8, device="cuda"), torch.tensor([3, 1], device="cuda")
    with pytest.raises(L.LMLossError):
        L.lmloss_vocab_create(torch.cuda.device_count(), 0)
    assert torch.equal(ops.embedding_forward(w, ids), w[ids])
    ops.close()


@pytest.mark.gpu
def test_first_call_on_a_side_stream_under_work_on_the_default_one():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    g = torch.Generator(device="cuda").manual_seed(1)
    z, s = torch.randn(8, 5003, device="cuda", generator=g), torch.zeros(2, 4, device="cuda")
    ids = torch.randint(0, 50, (5000,), device="cuda", generator=g)
    rows = torch.randint(-4, 5, (5000, 64), device="cuda", generator=g).float()
    want = torch.zeros(50, 64, device="cuda").index_add_(0, ids, rows)
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    reference = None
    for _ in range(4):
        for _ in range(8):
            a = a @ a * 1e-3                       # a few milliseconds queued on the default stream
        ops = VocabOps(0, max_tokens=5000, max_dim=64, max_rows=8, max_vocab=5003)
        step = ops.beam_step(z, s, stream=side)
        total = ops.embedding_backward(rows, ids, num_embeddings=50, stream=side)
        side.synchronize()
        if reference is None:
            reference = (step.tokens.clone(), step.scores.clone())
            top = (z.double() - z.double().logsumexp(1, keepdim=True)).view(2, -1).topk(4, dim=1)[1]
            assert torch.equal(step.parents.long() * 5003 + step.tokens, top)
        assert torch.equal(step.tokens, reference[0]) and torch.equal(step.scores, reference[1])
        assert torch.equal(total, want)
        ops.close()
