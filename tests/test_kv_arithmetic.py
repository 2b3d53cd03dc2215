"""CPU restatements, in numpy, of arithmetic that the attention kernels rely on."""
import numpy as np
import pytest

F = np.float32
MOST, COARSE = F(4096), F(2.0**24)


def _p(s, f, ref):
    """2^(f s - ref): one rounding, as a fused multiply-add; scores rounded first where the reference is coarse."""
    if abs(ref) >= COARSE:
        s, f = (s * f).astype(F), F(1)
    y = (s.astype(np.float64) * np.float64(f) - np.float64(ref)).astype(F)
    return np.exp2(y), s, f


def tile(s, f, ref):
    """A prompt row's tile of scores: (p, reference, rounds)."""
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        if ref == -np.inf:
            ref = F(s.max() * f)
        for rounds in (1, 2, 3):
            p, s, f = _p(s, f, ref)
            if not p.sum(dtype=F) > MOST:
                return p, ref, rounds
            ref = F(s.max() * f)
    raise AssertionError("the reference would move a third time")


@pytest.mark.parametrize("size", [1.0, 1e3, 1e6, 2.0**24, 1e8, 3e8, 1e9, 1e15, 1e30, 1e36])
def test_a_prompt_tile_moves_its_reference_once_at_most(size):
    rng = np.random.default_rng(int(np.log2(size)))
    for f in (F(0.1275), F(1.4427), F(3e-5)):
        for _ in range(300):
            s = (rng.standard_normal(64) * (size / f if size < 1e30 else size)).astype(F)
            for ref in (F(-np.inf), F(rng.standard_normal() * size), F(-size), F(size)):
                p, now, rounds = tile(s.copy(), f, ref)
                assert rounds <= 2 and np.all(np.isfinite(p))
                if rounds == 2 or ref == -np.inf:  # the reference is the largest score: p is 2^(half its spacing) at most
                    assert 0.49 < p.max() < 2.01 and np.argmax(p) in np.flatnonzero(s * f >= (s * f).max())
