"""The float64 oracle of the residual add with dropout (CPU): its generator
against published answers, its mask's shares, its gradients against differences."""
import numpy as np
import pytest

from oracle import dropout


def words(counter, key):
    return [int(v) for v in dropout.philox(np.array(counter, np.uint64), key)]


def test_generator_against_published_answers():
    """The known answers that come with the generator's paper (Random123)."""
    assert words([0, 0, 0, 0], (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert words([f, f, f, f], (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_places():
    """Column blocks of four, rows and the 64-bit offset each go where they are said to."""
    m = dropout.kept(3, 7, 0.5, 5, (9 << 32) + 8)
    for r in range(3):
        for c in range(7):
            w = words([c // 4, r, 8, 9], (5, 0))[c % 4]
            assert m[r, c] == (w >= 1 << 31)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1 - 2.0 ** -40])
def test_share_that_is_kept(p):
    """400000 independent draws: within five deviations."""
    n = 400 * 1000
    share = dropout.kept(400, 1000, p, 17, 3).mean()
    assert abs(share - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n)


def test_seeds_and_offsets_give_other_masks():
    a = dropout.kept(50, 64, 0.5, 1, 1)
    for other in (dropout.kept(50, 64, 0.5, 2, 1), dropout.kept(50, 64, 0.5, 1, 2),
                  dropout.kept(50, 64, 0.5, 1 + (1 << 32), 1), dropout.kept(50, 64, 0.5, -1, 1)):
        assert 0.4 < (a == other).mean() < 0.6


@pytest.mark.parametrize("name", ["x", "residual", "weight"])
def test_gradients_against_differences(name):
    g = np.random.default_rng(3)
    v = {"x": g.normal(size=(5, 9)), "residual": g.normal(size=(5, 9)), "weight": g.normal(size=9)}
    keep, dy, dro = dropout.kept(5, 9, 0.3, 1, 2), g.normal(size=(5, 9)), g.normal(size=(5, 9))
    way = g.normal(size=v[name].shape)

    def loss(step):
        u = {**v, name: v[name] + step * way}
        y, r = dropout.add_norm(u["x"], u["residual"], u["weight"], 0.5, 0.3, keep, 1e-5)
        return (y * dy).sum() + (r * dro).sum()

    _, r = dropout.add_norm(v["x"], v["residual"], v["weight"], 0.5, 0.3, keep, 1e-5)
    ref = dropout.add_norm_backward(r, v["weight"], dy, dro, 0.5, 0.3, keep, 1e-5)
    grad = ref[{"x": "dx", "residual": "dresidual", "weight": "dweight"}[name]]
    slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
    assert abs((grad * way).sum() - slope) <= 1e-7 * max(1.0, abs(slope))
