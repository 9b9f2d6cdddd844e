"""Head scales that the 4-bit cache's operators refuse before they touch a device (CPU)."""

import pytest

from test_kv4_refusals import P, _append, _shape, nsv  # noqa: F401 (nsv is a fixture)


@pytest.mark.parametrize("scales", [(P + 2, P), (P, P + 1), (P + 1, None), (None, P + 2)])
@pytest.mark.parametrize("rope", [True, False])
def test_append_scales_are_aligned(nsv, scales, rope):  # noqa: F811
    given = {} if rope else dict(q=None, q_out=None)
    assert _append(nsv, _shape(nsv), True, rope=rope, scales=scales, **given) == -4
    # (a null pointer is told first, as for the other arguments)
    assert _append(nsv, _shape(nsv), True, rope=rope, scales=scales, v=None, **given) == -1
