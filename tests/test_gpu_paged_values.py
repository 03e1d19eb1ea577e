"""GPU tests of the paged attention on the values at its borders: absent keys
beside rows that are not finite.  Cases and tolerances as in test_gpu_paged."""

import pytest

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_absent_window_keys_have_no_scale(kv, bad):
    """The last window tile of a query holds 2 keys; the 126 places behind
    them must not see the scales that an earlier tile left there, here of
    other requests whose scales are not finite."""
    c = Case([0] * 300, 1, 16, 130, kv, "fp8", seed=70)
    c.swa_scale[::2] = bad
    c.run().check([(b, 0) for b in range(1, 300, 2)])


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("W,window", [(0, "bf16"), (5, "fp8")])
def test_many_query_parts_per_cta(kv, W, window):
    """Some fourteen queries of one or two tiles per CTA: Q changes as often as the keys do."""
    lens = [(37 * b) % 190 for b in range(2100)]
    c = Case(lens, 1, 32, W, kv, window, seed=73)
    for _ in range(20):
        c.run()
    c.check([(b, 0) for b in range(0, 2100, 41)])
