"""What tree_attn may lose of a probability: 2^-16, not a bf16 rounding.

A bf16 value has 8 significant bits: rounding to it loses up to 2^-8 of a number, as much as the
outputs' own rounding.  The kernel multiplies V by probabilities in two bf16 pieces, so the rounding
that is left is the output's, and errors in proportion to sum p|v| have to be far smaller.

Inputs.  q and k hold -1, 0 and 1 and the scale is 2^-4, so scores are whole multiples of 2^-4, exact in
float; their spread in base two stays below 16.  V is any bf16.

Bound, for n keys, in units of mag = sum p|v|:
  pieces   upper piece cut off below 2^-7, the rest rounded: 2^-16, and 2^-20 from the factor 1 + 2^-20;
  p        rounded scale (2^-23 of 8), one fma (half a unit of 16: 2^-20), exp2 (2^-22): below 2^-19, once
           in the numerator and once in the sum;
  sum      a thread adds at most 64 keys of a tile, in four chains, then halves and parts: 2^-18;
  product  2 n / 16 steps of 16 keys, each taken as losing 2^-22 of all magnitudes: n 2^-25;
  the quotient: 2^-22.
The float terms are below 2^-17 + n 2^-25 + 2^-22, and with E their sum and the pieces'
    |out - ref| <= 2^-8 |ref| + (1 + 2^-8) E mag.
"""
import numpy as np
import pytest

from tests._gpu_util import f32_of_bf16

SCALE = 2.0 ** -4


def bf16(a):
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rounded(a):
    return f32_of_bf16(bf16(a)).astype(np.float64)


def cut(a):
    return (np.ascontiguousarray(a, np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)


class Case:
    """One cached request: `length` cached tokens and a chain of `nodes`, one cache head."""

    def __init__(self, seed, length, nodes, group, d):
        rng = np.random.default_rng(seed)
        n = length + nodes
        self.length, self.nodes, self.group, self.d = length, nodes, group, d
        self.q = rng.integers(-1, 2, (nodes, group, d)).astype(np.float64)
        self.k = rng.integers(-1, 2, (n, d)).astype(np.float64)
        self.v = rounded(rng.standard_normal((n, d)))
        may = np.arange(n) <= length + np.arange(nodes)[:, None]
        s = np.where(may[:, None], self.q @ self.k.T * SCALE, -np.inf)
        self.p = np.exp(s - s.max(-1, keepdims=True))       # [nodes, group, keys]
        assert (s.max(-1) - np.where(may[:, None], s, np.inf).min(-1)).max() * np.log2(np.e) < 16
        total = self.p.sum(-1, keepdims=True)
        self.ref, self.mag = self.p @ self.v / total, self.p @ np.abs(self.v) / total

    def excess(self, out):
        """The largest error over its bound."""
        n = self.length + self.nodes
        e = 2.0 ** -16 + 2.0 ** -20 + 2.0 ** -17 + n * 2.0 ** -25 + 2.0 ** -22
        return (np.abs(out - self.ref) / (2.0 ** -8 * np.abs(self.ref) + (1 + 2.0 ** -8) * e * self.mag)).max()

    def model(self, pieces):
        """The output with `pieces` of P (powers as the kernel's reference leaves them: up to 2^8)."""
        p = np.float32(self.p * 37.7)
        return rounded(pieces(p) @ self.v / p.astype(np.float64).sum(-1, keepdims=True))


CASES = [(length, nodes, group, d) for d in (64, 128, 256) for length, nodes, group in
         ((0, 7, 2), (20, 9, 3), (37, 1, 8), (90, 20, 5), (300, 16, 5))]


@pytest.mark.parametrize("length,nodes,group,d", CASES)
def test_the_bound_tells_two_pieces_from_less(length, nodes, group, d):
    c = Case(length + d, length, nodes, group, d)
    low = lambda p: np.float32(p * np.float32(1 + 2.0 ** -20)) - cut(p)
    assert c.excess(c.model(lambda p: cut(p) + rounded(low(p)))) <= 1
    assert c.excess(c.model(rounded)) > 1                                # one rounded piece
    assert c.excess(c.model(cut)) > 1                                    # the lower piece lost
    assert c.excess(c.model(lambda p: cut(p) + 0.5 * low(p))) > 1        # half of it


@pytest.mark.gpu
@pytest.mark.parametrize("length,nodes,group,d", CASES)
def test_probabilities_keep_sixteen_bits(length, nodes, group, d):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lossless_bit_weights_gb300 as w12
    from tests._gpu_util import to_dev16, to_np16
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    for seed in range(4):
        c = Case(length + d + 1000 * seed, length, nodes, group, d)
        blocks = max(1, -(-length // 16))
        kc, vc = np.zeros((2, blocks * 16, 1, d), np.uint16)
        kc[:length, 0], vc[:length, 0] = bf16(c.k[:length]), bf16(c.v[:length])
        cache = w12.KVCache(*[to_dev16(x.reshape(blocks, 16, 1, d)) for x in (kc, vc)])
        out, st = w12.tree_attn(to_dev16(bf16(c.q)), to_dev16(bf16(c.k[length:, None])), to_dev16(bf16(c.v[length:, None])),
                                cache, i32([list(range(blocks))]), i32([length]), i32(list(range(-1, nodes - 1))), scale=SCALE)
        assert int(st) == 0
        assert c.excess(f32_of_bf16(to_np16(out)).astype(np.float64)) <= 1
