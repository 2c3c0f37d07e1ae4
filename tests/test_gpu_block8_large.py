"""Products with more results than 2^32, in both types: every result exact."""
import pytest
import torch

import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_many_rows(out):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    rows, K, N, n = 1100003, 64, 8192, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-8, 9, s, generator=gen, device="cuda").float()  # noqa: E731
    a, w = whole(rows, K), whole(n, N, K)
    sa = torch.exp2(torch.randint(-2, 3, (1, rows), generator=gen, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 3, (n, N // 128, 1), generator=gen, device="cuda").float())
    split = 600001
    offsets = torch.tensor([0, split, rows], dtype=torch.int32, device="cuda")
    y = torch.full((rows, N), -7.0, dtype=out, device="cuda")
    mok.mok_block8_gemm(a.to(torch.float8_e4m3fn), sa, rows, K, w.to(torch.float8_e4m3fn), sw, N, y, offsets=offsets,
                        n_local=n)
    y2 = y.view(rows, N // 128, 128)
    for e, (first, end) in enumerate(((0, split), (split, rows))):
        for at in range(first, end, 1 << 16):
            to = min(at + (1 << 16), end)
            # 64 products of at most 64: whole numbers, and powers of two beside them
            want = (a[at:to] @ w[e].T).view(to - at, N // 128, 128) * sa[0, at:to, None, None] * sw[e, None]
            assert torch.equal(y2[at:to], want.to(out))
    del y, y2
    torch.cuda.empty_cache()
