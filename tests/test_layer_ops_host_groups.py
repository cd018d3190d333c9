"""A call of more than two groups of heads goes to the GPU as launches of two, and each launch's
groups share all of the CTAs: the gradient's workspace shows it, a row of partial sums per CTA."""
import pytest


def _group(heads, dgamma=True):
    return (16, 64, 64, 16, 64, 64, 16, 64, 64, 16, 16 if dgamma else 0, heads, False)


def _bytes(hm, *groups, rows=4096, dim=64):
    return hm.head_norm_rope_backward_workspace(hm.head_grad_list(groups), rows, dim)


@pytest.mark.parametrize("heads", [(20, 20, 20, 20), (40, 20, 20), (64, 8, 8), (32, 8, 8, 2), (1, 1, 1, 1), (3, 500, 1, 7)])
def test_a_pair_of_groups_has_all_ctas(hm, heads):
    g = [_group(h) for h in heads]
    assert _bytes(hm, *g) == _bytes(hm, *g[:2]) + _bytes(hm, *g[2:])


def test_groups_that_are_left_out_take_no_place(hm):
    a, b, c = _group(8), _group(4), _group(2)
    nothing, empty_sum = _group(0, False), _group(0)
    assert _bytes(hm, nothing, a, nothing, b) == _bytes(hm, a, b)
    assert _bytes(hm, a, nothing, b, c) == _bytes(hm, a, b) + _bytes(hm, c)
    # one without heads whose sum is wanted is in a launch, as the only one or beside another
    assert _bytes(hm, a, empty_sum, b, c) == _bytes(hm, a) + _bytes(hm, b, c)
    # and one whose sum is not wanted, too
    frozen = _group(8, False)
    assert _bytes(hm, a, frozen, b, c) == _bytes(hm, a, frozen) + _bytes(hm, b, c)
    assert _bytes(hm, a, frozen) < _bytes(hm, a)
    assert _bytes(hm, a, b, c, rows=0) == 0
