"""GPU tests of the scored route where the open groups' lanes keep fewer keys
than a token has picks, or little more: ordinary, distinct logits."""
import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("E,k,G,top_groups,T", [
    (512, 12, 8, 1, 2051), (512, 9, 8, 1, 2051), (512, 12, 8, 2, 2051), (512, 6, 16, 1, 2051), (512, 5, 16, 1, 2051),
    (256, 9, 16, 2, 2051), (512, 12, 4, 1, 2051),                  # four tokens to a wave
    (4092, 6, 33, 1, 70), (2640, 5, 40, 1, 70), (2640, 9, 40, 2, 70), (128, 16, 8, 1, 2051)])
def test_fewer_keys_than_picks(E, k, G, top_groups, T, score):
    rng = np.random.default_rng(E + k + G)
    for with_bias, top2 in ((True, True), (False, False), (True, False)):
        l = rng.normal(size=(T, E)).astype(np.float32)
        b = (0.1 * rng.normal(size=E)).astype(np.float32) if with_bias else None
        want, gate, load, gaps = ref.route_and_gaps(l, score, k, b, G, top_groups, top2, True, 2.5)
        clear = gaps >= 2.0 ** -45
        assert clear.mean() > 0.99
        r = mok.mok_router_desc(n_experts=E, top_k=k, score=score, n_groups=G, top_groups=top_groups,
                                group_rule=int(top2), renorm=1, scale=2.5)
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        got = torch.full((T, k), float("nan"), device="cuda")
        mok.mok_route_scored(r, torch.from_numpy(l).cuda(), T, idx, got, bias=None if b is None else torch.from_numpy(b).cuda())
        assert np.array_equal(idx.cpu().numpy()[clear], want[clear])
        # (2 |x| + 96) 2^-24 of the gate, |x| at most 12 here
        err = np.abs(got.double().cpu().numpy() - gate)[clear]
        assert np.all(err <= 120 * 2.0 ** -24 * gate[clear])
