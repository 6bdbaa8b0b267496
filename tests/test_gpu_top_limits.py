"""Top alternatives of every number up to the limit: the sizes at which the
call's shared memory is just below and just above what a launch gets without
asking for more, and two host threads whose calls ask for different amounts."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (bf16, vocabulary, rows, top k): 48 KB of dynamic shared memory less a few
# hundred bytes, for one block a row and for clusters
EDGES = [(True, 65536, 250, 200), (True, 65536, 250, 201), (True, 128256, 4, 155), (True, 128256, 4, 156),
         (True, 128256, 100, 182), (True, 50257, 400, 220), (True, 1000, 3, 226), (False, 65536, 250, 197),
         (False, 128256, 4, 154), (False, 32000, 8, 156), (False, 50257, 400, 215), (False, 1000, 3, 226)]

CHILD = """
import sys, torch
sys.path[:0] = ["tests"]
import float8_mixed_precision_gb300 as f8
import ops_reference as ref
for bf, vocab, rows, k in %r:
    g = torch.Generator(device="cuda:0").manual_seed(k)
    z = (torch.randn((rows, vocab), generator=g, device="cuda:0") * 3).to(torch.bfloat16 if bf else torch.float32)
    lse, ids, top = f8.f8_token_logprobs(z, top_k=k)[2:]
    r = ref.token_logprobs(z, None, 1.0, k)
    assert torch.equal(ids.long(), r["top_ids"]), (bf, vocab, rows, k)
    ref.check(top, r["top_logp"], r["b_top"], str((bf, vocab, rows, k)))
assert f8.f8_last_device_status() == 0
print("all right")
"""


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


def test_every_size_is_taken(f8):
    """In a process of its own, in which no larger call came before."""
    r = subprocess.run([sys.executable, "-c", CHILD % (EDGES,)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "all right" in r.stdout, (r.stdout + r.stderr)[-2000:]


def test_two_threads(f8):
    """Two host threads whose calls need different amounts of shared memory
    above 48 KB: 20,000 C calls each, none of them refused."""
    z = torch.randn((4, 131072), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    call = f8.lib().f8_token_logprobs
    start, refused, got = threading.Barrier(2), [], {}

    def work(k):
        ids = torch.zeros((4, k), dtype=torch.int32, device=DEV)
        top = torch.zeros((4, k), device=DEV)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        args = (z.data_ptr(), f8.F8_BF16, 4, 131072, 131072, None, 1.0, k, None, None, None, ids.data_ptr(),
                top.data_ptr(), stream.cuda_stream)
        start.wait()
        refused.extend(k for _ in range(20000) if call(*args) != 0)
        stream.synchronize()
        got[k] = ids

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in (256, 170)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not refused, (len(refused), set(refused))
    for k, ids in got.items():
        assert torch.equal(ids.long(), ref.token_logprobs(z, None, 1.0, k)["top_ids"])
    assert f8.f8_last_device_status() == 0
