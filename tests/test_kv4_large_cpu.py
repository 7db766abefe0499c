"""What the tests of large calls put in place of the oracle's loops."""
import numpy as np

from oracle import kv4_oracle as K
from tests.test_gpu_kv4_large import places, quantize


def test_the_places_are_the_oracles():
    rng = np.random.default_rng(0)
    for trial in range(20):
        seqs, page, pages, width = 9, 16, 12, 3
        new = rng.integers(0, 12, seqs)
        lengths = np.maximum(new + rng.integers(-6, 50, seqs), 0)
        starts = np.concatenate([[0], np.cumsum(new)])
        table = rng.integers(-1, pages + 1, (seqs, width))
        tokens = int(starts[-1]) + 4
        kind, at, place = places(starts, lengths, table, page, pages, tokens)
        for r, want in enumerate(K.places(starts, lengths, table, page, pages, tokens)):
            got = (0, 1, 2, 3)[kind[r]]
            assert {"before": 0, "nowhere": 2, None: 3}.get(want if not isinstance(want, tuple) else 1, 1) == got
            if isinstance(want, tuple):
                assert want == (at[r], place[r])


def test_the_codes_are_the_oracles():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 2, 64)) * np.exp(5 * rng.standard_normal((50, 2, 1)))
    x[3], x[4, 0, :32], x[5] = 0, 1e-44, np.repeat(np.arange(-16, 16) / 4.0, 2)
    x[6, 1, :32], x[7, :, ::2] = 6.0, 1.5 * 2.0 ** 100
    for a, b in zip(quantize(x), K.quantize(x)):
        assert np.array_equal(a, b)
