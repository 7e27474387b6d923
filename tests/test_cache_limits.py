"""Ends of the rotation and cache calls' ranges that need no GPU: refusals, calls with nothing to do."""
import pytest

from test_cache_abi import A, INVALID, L, attn, batch, cache  # noqa: F401


@pytest.mark.parametrize("kind,most,over", [(0, 2e38, 3e38), (1, 3.9e17, 4.1e17)])
def test_scales_past_the_kernels_numbers_are_refused(L, kind, most, over):  # noqa: F811
    """The scale goes in times log2(e), with 4 bits times 2^69 as well; every smaller one is taken."""
    c = cache(kind=kind, k_scales=A, v_scales=A)
    empty = batch(num_tokens=0, cu_new=A)  # nothing to do: returns behind the checks
    assert attn(L, c=c, b=empty, scale=over) == INVALID
    for scale in (most, 1.0, 1e-30, 1e-38, 1e-45):
        assert attn(L, c=c, b=empty, scale=scale) == 0
