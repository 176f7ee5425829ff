"""The attention block's operators where the order of the kernels' steps, the
range of the number formats or the limits of the arguments matter. Reference
and tolerances as in test_gpu_paged.py unless a test says otherwise."""
import pytest
import torch

from test_gpu_paged import KINDS, Paged, pkg  # noqa: F401  (pkg is a fixture)

pytestmark = pytest.mark.gpu

RAGGED = [70 + 37 * i % 59 for i in range(64)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([256] * 32, [256] * 32),        # prompts from an empty cache: up to 7 items a CTA, one tile of keys in the first ones
    ([512] * 8, [512] * 8),          # 2 to 4 pieces a CTA, one-tile items after split ones
    (RAGGED, RAGGED),                # nothing but one-tile items, of 280 to 512 rows
    ([100 if i % 3 else 130 for i in range(48)], [100 if i % 3 else 700 + 90 * i for i in range(48)]),  # and between longer ones
])
def test_attend_many_pieces_of_a_cta(pkg, new, lens, d, dtype, cache):  # noqa: F811
    """CTAs of the many-row kernel walk several items one after the other; the size of the queries changes by powers of
    two between the row tiles and sequences, so that a row taken with another item's scale shows."""
    s = Paged(pkg, new, lens, heads=32, kv_heads=8, d=d, dtype=dtype, cache=cache, page=32, seed=len(new))
    size = torch.cat([2.0 ** (-3 * ((5 * b + torch.arange(n) // 64) % 4)) for b, n in enumerate(new)]).cuda()
    q = (s.rows(32, 1.5).float() * size[:, None, None]).to(dtype)
    out = s.check(q)
    for _ in range(5):
        assert torch.equal(s.layer.attend(s.cache, s.batch, q), out)
