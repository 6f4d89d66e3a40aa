"""draft_accept's binding: which row layouts of the probabilities it hands to the library.

The library reads rows that lie one even step apart, at least V elements. A step below V
(broadcast or overlapping rows) must be refused, never replaced: the kernel would read past
the tensor. Host stand-ins that claim to be on the GPU; no CUDA call.
"""
import pytest

torch = pytest.importorskip("torch")

import lfm2_gated_short_gb300 as sc  # noqa: E402

V = 100


class Fake:
    """What _prob_rows looks at, of a host tensor."""

    is_cuda, device = True, "cuda:0"

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, t.shape

    def stride(self):
        return self.t.stride()

    def data_ptr(self):
        return self.t.data_ptr()


def rows(t):
    return sc._prob_rows(Fake(t), "target", torch.float32, tuple(t.shape))


def last_element(t):
    """The element past the last one that rows of V at the returned step reach, from the start."""
    N, n, _ = t.shape
    return (N * n - 1) * rows(t)[1] + V


BASE = torch.zeros(40 * V)
BROADCAST = {
    "one row for all": BASE[:V].expand(3, 4, V),
    "one row for all positions": BASE[:V].view(1, 1, V).expand(1, 4, V),
    "one row for all sequences": BASE[:V].view(1, 1, V).expand(3, 1, V),
    "a row a sequence": BASE[:3 * V].view(3, 1, V).expand(3, 4, V),
    "a row a position": BASE[:4 * V].view(1, 4, V).expand(3, 4, V),
    "overlapping rows": BASE.as_strided((3, 4, V), (40, 10, 1)),
    "overlapping rows of one sequence": BASE.as_strided((1, 4, V), (400, V - 1, 1)),
    "overlapping sequences of one row": BASE.as_strided((3, 1, V), (V - 1, V, 1)),
}


@pytest.mark.parametrize("name", BROADCAST)
def test_rows_closer_than_their_width_are_refused(name):
    with pytest.raises(ValueError, match="rows"):
        rows(BROADCAST[name])


@pytest.mark.parametrize("shape,stride,step", [
    ((3, 4, V), (4 * V, V, 1), V),            # contiguous
    ((3, 4, V), (4 * 120, 120, 1), 120),      # sliced from wider rows
    ((1, 4, V), (7, 130, 1), 130),            # one sequence: its own step is never taken
    ((3, 1, V), (130, 5, 1), 130),            # one row a sequence: nor is the row's
    ((1, 1, V), (0, 0, 1), V),                # one row: any step
    ((1, 1, V), (1000, 1000, 1), V),
    ((0, 4, V), (0, 0, 1), V),                # no rows
    ((3, 0, V), (0, 0, 1), V),
])
def test_rows_one_even_step_apart_are_taken(shape, stride, step):
    t = BASE.as_strided(shape, stride)
    p, s = rows(t)
    assert (p, s) == (t.data_ptr(), step)
    if t.numel():
        assert last_element(t) <= BASE.numel()


def test_uneven_or_scattered_rows_are_refused():
    for stride in ((500, 100, 1), (400, 100, 2)):
        with pytest.raises(ValueError, match="rows"):
            rows(BASE.as_strided((2, 4, V), stride))
