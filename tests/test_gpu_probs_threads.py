"""idx_logit_probs called by two host threads at once, with rows that take different amounts of shared memory."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
CALLS = 20000


@pytest.mark.parametrize("dtype,code", [(torch.float32, 2), (torch.bfloat16, 0)])
def test_two_threads_with_small_and_large_rows(lib, dtype, code):
    """Straight to the C entry, which runs without the interpreter's lock: each call is accepted, and the last ones are right."""
    entry = lib.load_library().idx_logit_probs
    gate, refused, outputs = threading.Barrier(2), [], {}
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    rows = {vocab: torch.randn(1, vocab, device="cuda").to(dtype) for vocab in (100, 200_003)}
    want = {vocab: torch.softmax(x.double(), 1) for vocab, x in rows.items()}
    torch.cuda.synchronize()

    def work(vocab):
        stream, probs = torch.cuda.Stream(), torch.empty(1, vocab, device="cuda")
        args = [rows[vocab].data_ptr(), vocab, code, vocab, 1, cu.data_ptr(), 1, *[None] * 5, 0, *[None] * 5, 0, None, 0, probs.data_ptr(), vocab, None, None,
                stream.cuda_stream]
        gate.wait(60)
        refused.append(sum(entry(*args) != 0 for _ in range(CALLS)))
        stream.synchronize()
        outputs[vocab] = probs

    threads = [threading.Thread(target=work, args=(vocab,)) for vocab in rows]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == [0, 0]
    for vocab, p in outputs.items():
        # 4 d + 128 units of 2^-24, d at most 12 between normal values
        assert ((p.double() - want[vocab]).abs() <= want[vocab] * 2.0**-24 * (4 * 12 + 128)).all()
