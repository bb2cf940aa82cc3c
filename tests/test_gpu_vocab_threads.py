"""Two host threads, each with its own vocabulary handle and stream, call the operators at the same
time: the sorts raise launch limits that are the process's, the results are those of the calls alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def make(seed, T, V, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, K = 3, 4
    return dict(ids=torch.randint(0, V, (T,), device="cuda", generator=g),
                rows=torch.randn(T, D, device="cuda", generator=g).to(dtype),
                base=torch.randn(V, D, device="cuda", generator=g),
                z=torch.randn(B * K, V, device="cuda", generator=g).to(dtype),
                s=-torch.rand(B, K, device="cuda", generator=g) * 10,
                kv=torch.randn(B * K, 5, 33, device="cuda", generator=g).to(dtype))


def call(ops, x, stream=None):
    step = ops.beam_step(x["z"], x["s"], num_candidates=4, stream=stream)
    moved, = ops.beam_reorder([x["kv"]], step.parents, stream=stream)
    look = ops.embedding_forward(x["base"], x["ids"], scale=0.5, out_dtype=x["rows"].dtype, stream=stream)
    whole = ops.embedding_backward(x["rows"], x["ids"], num_embeddings=x["base"].shape[0], stream=stream)
    return step.scores, step.parents, step.tokens, step.lse, moved, look, whole


def test_two_threads_two_handles():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    # one sorts in a cluster, the other with aligned and unaligned rows by counting or in passes
    sizes = [(9000, 5001, 96, torch.bfloat16), (140000, 3000, 17, torch.float32), (3000, 9000, 33, torch.float16)]
    inputs = [make(i, *s) for i, s in enumerate(sizes)]
    refs = []
    for x in inputs:
        ops = VocabOps(0, max_tokens=140000, max_dim=128, max_rows=64, max_vocab=1 << 14)
        refs.append(call(ops, x))
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        ops.close()
    errors, start = [], threading.Barrier(len(sizes))

    def work(i):
        try:
            torch.cuda.set_device(0)
            ops = VocabOps(0, max_tokens=140000, max_dim=128, max_rows=64, max_vocab=1 << 14)
            stream = torch.cuda.Stream()
            start.wait(60)
            for _ in range(20):
                got = call(ops, inputs[i], stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, refs[i])):
                errors.append(f"thread {i}: other bits than alone")
            if ops.device_error() != 0:
                errors.append(f"thread {i}: device error")
            ops.close()
        except Exception as e:  # noqa: BLE001
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
