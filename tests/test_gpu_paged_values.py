"""GPU tests of the paged attention on the values at its borders: absent keys
beside rows that are not finite.  Cases and tolerances as in test_gpu_paged."""

import pytest

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_absent_window_keys_have_no_scale(bad):
    """The last window tile of a query holds 2 keys; the 126 places behind
    them must not see the scales that an earlier tile left there, here of
    other requests whose scales are not finite."""
    c = Case([0] * 300, 1, 16, 130, "fp4", "fp8", seed=70)
    c.swa_scale[::2] = bad
    c.run().check([(b, 0) for b in range(1, 300, 2)])
