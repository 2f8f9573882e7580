"""The loss's gradients with the vocabulary in several pieces, in the forms that many rows do
not reach: few rows with a target among many (G in two parts whose sums add up over pieces),
sums of dh both over pieces and in parts, and several tiles of dims.
Definition and tolerances as in test_gpu_lm_loss."""
import pytest

from test_gpu_lm_loss import check, launch, make, reference

pytestmark = pytest.mark.gpu


def some_targets(t, keep, seed):
    """All but `keep` targets taken out."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t[torch.randperm(len(t), generator=g, device="cuda")[keep:]] = -1
    return t


# 20001 rows: two pieces, of 34 and 33 tiles of 256 words.  9000: five, each in two parts for dh.  300
# rows and 700001 words: two pieces in 38 parts.  D = 264 and 520: tiles of dims that end inside.
@pytest.mark.parametrize("n,D,V,keep", [(20001, 64, 17000, 1), (20001, 64, 17000, 100), (20001, 72, 17000, 128), (20001, 64, 17000, 129),
                                        (20001, 264, 17000, 90), (9000, 64, 151936, 128), (9000, 64, 151936, 300),
                                        (300, 72, 700001, 100), (300, 72, 700001, 300)])
def test_few_targets_among_many_rows(padoc_lib, n, D, V, keep):
    h, w, t, d = make(n, D, V, seed=n + keep)
    t = some_targets(t, keep, 1)
    check(launch(h, w, t, d), *reference(h, w, t, d))


@pytest.mark.parametrize("n,D,V", [(20001, 264, 17000), (20001, 520, 17153), (9000, 72, 151936)])
def test_pieces_with_parts_and_tiles_of_dims(padoc_lib, n, D, V):
    h, w, t, d = make(n, D, V, seed=n + D, masked=0.3)
    check(launch(h, w, t, d), *reference(h, w, t, d))


@pytest.mark.parametrize("which", ["dh", "dw"])
def test_one_gradient_of_few_targets(padoc_lib, which):
    import torch
    h, w, t, d = make(20001, 64, 17000, seed=2)
    t = some_targets(t, 100, 3)
    both = launch(h, w, t, d)
    one = launch(h, w, t, d, dh=which == "dh", dw=which == "dw")
    i = 2 if which == "dh" else 3
    assert torch.equal(both[i], one[i])
    again = launch(h, w, t, d)
    for a, b in zip(both, again):
        assert torch.equal(a, b)
