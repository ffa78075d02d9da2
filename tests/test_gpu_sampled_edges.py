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


@pytest.mark.parametrize("V", [2, 3, 7])
def test_greedy_requests_whose_drafter_was_sure(w12, V):
    """At temperature 0 the rule is the same: a token that the drafter had none of any more is passed over, and where
    it was certain of the target's token, a refused sibling leaves nothing."""
    rng = np.random.default_rng(V)
    for seed in range(6):
        p = Problem(seed, [6] * 100, V, temperature=None, sd=8.0, shape="star" if seed % 2 else "tree")
        p.T = np.zeros(100, np.float32)
        p.draft = rng.integers(-1, V + 1, p.draft.shape).astype(np.int32)
        if seed < 4:                     # q of one token at a time, with rounding's leavings on the others
            sure = rng.integers(0, V, len(p.draft))
            p.probs = (p.probs * np.float32(1e-8)).astype(np.float32)
            p.probs[np.arange(len(sure)), sure] = 1.0
        p.check(w12)


@pytest.mark.parametrize("q,draft,length", [
    ([1.0, 1e-8, 0.0], [0, 1], 0),            # after the first there is nothing the drafter could have drawn
    ([1e-9, 1.0, 0.0], [0, 1], 0),            # nothing is left of p
    ([0.0, 1.0, 0.0], [0, 1], 1),             # a token with q = 0 changes nothing
    ([0.5, 0.25, 0.25], [0, 2, 1], 1), ([0.5, 0.25, 0.25], [0, 0, 1], 1), ([0.5, 0.25, 0.25], [0, 3, -1, 1], 1),
    ([0.7, 0.7, 0.0], [0, 1], 0),             # u q is above what is left
    ([0.6, 0.6, 0.0], [1, 0], 1)])
def test_greedy_child(w12, q, draft, length):
    n = len(draft) + 1
    logits = f32(np.tile([0.0, 5.0, 1.0], (n, 1)))
    got, path, bonus, status = w12.tree_verify_sampled(
        logits, i32([-1] + [0] * (n - 1)), i32([0] + draft), f32(np.full(n, 0.875)), f32([0.5]),
        draft_probs=f32(np.tile(q, (n, 1))), temperature=f32([0.0]))
    assert (int(status), int(got), int(bonus)) == (0, length, 1)
