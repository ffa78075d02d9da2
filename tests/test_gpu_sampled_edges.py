"""tree_verify_sampled at the ends of its documented ranges: against the definition in 64 bits of test_gpu_sampled.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_sampled import Problem, f32, i32, w12  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T", [1.0, 1e30, np.inf])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("counts,V", [([1, 1], 5000), ([4, 6, 1], 3001), ([2] * 200, 60001)])
def test_infinite_logits_at_any_temperature(w12, T, probs, counts, V):
    """+inf tokens share p evenly, wherever they stand in the row and however flat the others are."""
    p = Problem(3, counts, V, probs=probs, temperature=None)
    rng = np.random.default_rng(4)
    M = sum(counts)
    for m in range(M):
        p.logits[m, rng.integers(V // 2, V, m % 4)] = np.inf
    p.logits[0, -1] = np.inf
    for m in range(1, M, 3):  # drafts that may be taken
        best = np.flatnonzero(np.isinf(p.logits[m - 1]))
        if len(best):
            p.draft[m] = best[0]
    p.T = np.full(len(counts), T, np.float32)
    p.check(w12)


def test_offsets_of_a_single_node(w12):
    """Offsets that fall make all requests out of range, with one node too; requests without nodes beside the one that
    has it are in order."""
    p = Problem(5, [1], 900, temperature=None)
    want = p.want()
    for off, whose in (([0, 1, 0, 1], None), ([0, 1, 1, 0], None), ([1, 0, 1, 1], None), ([0, 0, 1, 1], 1), ([0, 1, 1, 1], 0),
                       ([0, 0, 0, 1], 2)):
        length, path, bonus, status = w12.tree_verify_sampled(
            f32(p.logits), i32([-1]), i32([0]), f32([0.0]), f32(np.repeat(p.ub, 3)), req_offsets=i32(off))
        assert int(status) == (whose is None), off
        assert length.tolist() == [0 if r == whose else -1 for r in range(3)], off
        assert bonus.tolist() == [want[2][0] if r == whose else -1 for r in range(3)], off
        if whose is not None:
            assert path.tolist() == [0]


FIRST_CALLS = """
import threading, torch
import lossless_bit_weights_gb300 as w12
w12.lib()
g = torch.Generator(device="cuda").manual_seed(0)
V, n = 40000, 8
logits = 3 * torch.randn((n, V), generator=g, device="cuda")
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
parent, draft = i32([-1, 0, 0, 1, 1, 2, 3, 4]), torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
u, ub = torch.rand(n, generator=g, device="cuda"), torch.rand(1, generator=g, device="cuda")
streams, out, wait = [torch.cuda.Stream() for _ in range(16)], [None] * 16, threading.Barrier(16)
torch.cuda.synchronize()

def call(i):
    with torch.cuda.stream(streams[i]):
        ws = w12.Workspace()
        streams[i].synchronize()
        wait.wait()
        out[i] = [w12.tree_verify_sampled(logits, parent, draft, u, ub, ws=ws) for _ in range(20)]

threads = [threading.Thread(target=call, args=(i,)) for i in range(16)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
results = {tuple(tuple(x.tolist()) for x in r) for o in out for r in o}
assert len(results) == 1 and next(iter(results))[3] == (0,), results
"""


def test_first_calls_of_many_threads(w12):
    """The process's first calls come from 16 host threads at once, each on a stream and workspace of its own."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
