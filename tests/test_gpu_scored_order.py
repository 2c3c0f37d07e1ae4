"""GPU tests of the scored route's order where choice values are 2^-48 to 2^-46
of themselves apart: saturated sigmoids with a bias that is the same for all.

Both sides evaluate s = 1 / (1 + exp(-l)) and c = s + bias in fp64: exp(-l) is
below 2^-34 here, so its error is far below the rounding of 1 + exp(-l) (2^-53),
of the reciprocal (2^-54 below 1) and of the sum (at most 2^-52): less than
2^-51 of c in all on each side, two of which cannot turn round what is 2^-48
apart."""
import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
E, LOW, HIGH = 16, 3, 12


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _rows():
    """A row for each pair of logits from 24 to 40 in steps of a quarter, the smaller one at the lower id."""
    values = np.arange(24.0, 40.25, 0.25)
    small, large = np.triu_indices(len(values), 1)
    l = np.full((len(small), E), -8.0) - 0.5 * np.arange(E)
    l[:, LOW], l[:, HIGH] = values[small], values[large]
    return l.astype(np.float32)


@pytest.mark.parametrize("bias", [0.0, 0.25, -2.0])
@pytest.mark.parametrize("k,G,top_groups", [(1, 1, 1), (2, 1, 1), (15, 1, 1), (1, 4, 2), (2, 4, 2)])
def test_saturated_sigmoids_in_their_order(k, G, top_groups, bias):
    l = _rows()
    T = len(l)
    assert T > 2048                                     # all of them: many tokens; a thousand: few
    b = np.full(E, bias, np.float32)
    want, _, _, gaps = ref.route_and_gaps(l, ref.SIGMOID, k, b, G, top_groups)
    first = np.abs(np.diff(ref.scores(ref.clean(l), ref.SIGMOID)[:, [LOW, HIGH]] + bias))[:, 0] / max(1 + bias, -bias - 1)
    clear = gaps >= 2.0 ** -48
    assert clear.sum() > T // 2 and np.sum(clear & (first < 2.0 ** -46)) > 20
    r = mok.mok_router_desc(n_experts=E, top_k=k, score=mok.MOK_SCORE_SIGMOID, n_groups=G, top_groups=top_groups,
                            group_rule=mok.MOK_GROUP_MAX, renorm=0, scale=1.0)
    x, bt = torch.from_numpy(l).cuda(), torch.from_numpy(b).cuda()
    for n in (T, 1000):
        for at in range(0, T, n):
            rows = slice(at, min(at + n, T))
            m = rows.stop - at
            idx = torch.full((m, k), -7, dtype=torch.int32, device="cuda")
            gate = torch.empty(m, k, device="cuda")
            mok.mok_route_scored(r, x[rows], m, idx, gate, bias=bt)
            assert np.array_equal(idx.cpu().numpy()[clear[rows]], want[rows][clear[rows]]), (n, at)
