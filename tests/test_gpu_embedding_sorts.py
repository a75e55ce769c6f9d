"""The embedding's gradient where tokens are sorted: through global memory, and by several
threads that come to it at once."""
import subprocess
import sys

import pytest

from test_gpu_embedding import check_gradient, ids_like, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["uniform", "half", "zipf"])
@pytest.mark.parametrize("n", [65535, 65536, 65537, 131072, 250001])
@pytest.mark.parametrize("v", [300, 32000, 300000])
def test_many_tokens(n, v, kind):
    """More than 65536 tokens do not fit in a cluster's shared memory; one, two and three passes over the ids."""
    gy = table_of(n, 8, "bf16", n)
    check_gradient(gy, ids_like(kind, n, v, n), v, accumulate=kind == "zipf", padding=0 if kind == "half" else None)


def test_a_million_tokens():
    n, v = (1 << 20) + 33, 128256
    gy = table_of(n, 4, "fp32", 2)
    check_gradient(gy, ids_like("zipf", n, v, 3), v, id_type="int32")


FIRST_CALLS = """
import threading, torch
import linear_cross_entropy_03_gb300 as flce
sizes = [1500, 1500, 5000, 5000, 70000, 70000]
made = []
for k, n in enumerate(sizes):
    gen = torch.Generator(device="cuda").manual_seed(k)
    made.append((torch.randn(n, 64, generator=gen, device="cuda"), torch.randint(0, 400, (n,), generator=gen, device="cuda")))
torch.cuda.synchronize()
got, start = [None] * len(sizes), threading.Barrier(len(sizes))
def calls(k):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[k] = [flce.embedding_backward(*made[k], 400)["grad_weight"] for _ in range(5)]
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=calls, args=(k,)) for k in range(len(sizes))]
[t.start() for t in threads]
[t.join() for t in threads]
for k in range(len(sizes)):
    want = flce.embedding_backward(*made[k], 400)["grad_weight"]
    assert all(torch.equal(g, want) for g in got[k]), k
print("same")
"""


def test_first_calls_of_a_process_from_several_threads():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
