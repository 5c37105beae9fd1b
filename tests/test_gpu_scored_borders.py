"""The scored router where a choice or a weight hangs on the last bits of a score, against its 64-bit
definition."""
import itertools

import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import ops_oracle as O
from test_gpu_scored import BF, F32, biases, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def randn(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape)))


# ------------------------------------------------------------------------------ choice of groups
# groups of 2, 7, 8, 15, 20 and 32 experts: a share of a lane, lanes next to each other, neither
GROUPED = [(1, 8, 2, 4, 2), (40, 128, 8, 16, 3), (300, 160, 6, 8, 3), (4000, 160, 6, 8, 3),
           (300, 256, 8, 8, 4), (200, 56, 5, 8, 4), (700, 60, 4, 4, 1), (100, 960, 8, 64, 9)]


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T,E,k,groups,top", GROUPED)
def test_groups_of_peaked_logits(handle, T, E, k, groups, top, best):
    """Most scores are far below the largest one: groups that differ only in those are still told
    apart, whether weights are renormalised or not."""
    for renorm, bias in itertools.product((True, False), (None, biases(E))):
        for dtype, size in ((F32, 10.0), (BF, 10.0), (F32, 30.0)):
            check(handle, (size * randn(T, E)).to(dtype), bias, k, "softmax", renorm, 2.5, groups, top,
                  best)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T,E,k,groups,top", GROUPED)
def test_groups_of_nearly_equal_logits(handle, T, E, k, groups, top, best):
    """Scores within 1e-10 of each other: one step of the whole numbers that stand for them."""
    for score, renorm, base in itertools.product(("softmax", "sigmoid"), (True, False), (0.0, 1e-6)):
        check(handle, base + 1e-9 * randn(T, E), None, k, score, renorm, 1.0, groups, top, best)


@pytest.mark.parametrize("renorm", [True, False])
def test_groups_whose_best_scores_are_all_small(handle, renorm):
    """One logit far above all others: the second group is the one of the next largest logit, not the
    first of those whose scores are tiny."""
    x = torch.tensor([[40.0, 0, 1, 0, 2, 0, 10, 0], [0.0, 1, 2, 3, 90, 4, 6, 5]])
    for dtype, T in itertools.product((F32, BF), (1, 3, 300)):
        check(handle, x.repeat(T, 1).to(dtype), None, 2, "softmax", renorm, 1.0, 4, 2, 1)


# ------------------------------------------------------------------------------------- weights
def weights(handle, x, bias, k, **kw):
    args = dict(score="softmax", renorm=True, scale=1.0, groups=1, top=1, best=1) | kw
    return run(handle, x, bias, k, **args)[:2]


@pytest.mark.parametrize("below", [600.0, 700.0, 708.5, 709.5, 710.0, 720.0, 740.0, 744.0, 745.0, 746.0,
                                   1000.0])
def test_renormalised_weights_far_below_an_expert_left_out(handle, below):
    """The bias closes the expert of the largest logit, and the chosen scores are as small as 64 bits
    hold; a weight is 0 only where they are 0."""
    inf = float("inf")
    for dtype, T in itertools.product((F32, BF), (1, 20, 300)):
        x = torch.tensor([[0.0, -below]]).to(dtype)
        # as bf16 rounds it
        check(handle, x.repeat(T, 1), torch.tensor([-inf, 0.0]), 1, "softmax")
        check(handle, x.repeat(T, 1), torch.tensor([-inf, 0.0]), 1, "softmax", False)
    # two chosen ones: their weights are those of the difference of their logits
    for gap in (0.0, 0.5, 3.0):
        x = torch.tensor([[0.0, -float("inf"), -below, -below - gap]])
        for bias, kw in ((torch.tensor([-inf, 0.0, 0.0, 0.0]), {}),
                         (torch.tensor([-2.0, 0.0, 0.0, 0.0]), dict(groups=2, top=1)),
                         (torch.tensor([-2.0, 0.0, 0.0, 0.0]), dict(groups=2, top=1, best=2))):
            w, e = weights(handle, x, bias, 2, **kw)
            assert sorted(e[0].tolist()) == [2, 3] and (gap == 0.0 or below > 744 or int(e[0, 0]) == 2)
            # e^-745.13 is the least that rounds to a value other than 0
            want = torch.softmax(x[0, e[0].long()].double(), -1) if below < 745.13 else torch.zeros(2)
            O.assert_close(w[0], want, 1e-12 * want, f"{below} {gap} {kw}", half=O.U32)


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoids_next_to_the_least(handle, renorm):
    """Scores down to 1 / (1 + e^709.78), behind which e^-x has no 64-bit value and the score is 0."""
    rows = [[-709.5] * 6, [-720.0, -709.5, -709.25, -800.0, -709.0, -708.75],
            [-709.78271484375, -709.78265380859375, -709.75, -720.0, -709.78265380859375, -1000.0],
            [-1000.0, -710.0, -709.0, -709.03125, -709.0625, -708.0],
            [-800.0, -750.0, -720.0, -711.0, -710.0, -709.78271484375]]
    for bias, k in itertools.product((None, torch.zeros(6)), (1, 2, 3, 6)):
        check(handle, torch.tensor(rows), bias, k, "sigmoid", renorm)
        check(handle, torch.tensor(rows * 100), bias, k, "sigmoid", renorm)
        if k <= 4:
            for best in (1, 2):
                check(handle, torch.tensor(rows), bias, k, "sigmoid", renorm, 1.0, 3, 2, best)


@pytest.mark.parametrize("renorm", [True, False])
def test_an_infinite_logit_next_to_the_largest_finite_one(handle, renorm):
    """Only other infinite logits share the weight with it, also where the bias leaves them out."""
    inf, most = float("inf"), torch.finfo(F32).max
    rows = [[most, inf, 1.0, most, inf, 0.0], [most, most, 0.0, -most, 1e38, most], [inf, -inf, most, 0, 1, 2]]
    for bias, k in itertools.product((None, torch.zeros(6), torch.tensor([0, .5, 0, -.5, 0, .25]),
                                      torch.tensor([0, -inf, 0, 0, -inf, 0])), (1, 3, 4)):
        check(handle, torch.tensor(rows), bias, k, "softmax", renorm)
        for best in (1, 2):
            check(handle, torch.tensor(rows), bias, k, "softmax", renorm, 1.0, 3, 2, best)
