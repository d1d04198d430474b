"""More CPU tests of the host side of the operators over 8-bit caches and pages.
Every call below returns before it touches the GPU."""
from test_kv_host import EINVAL, ENOSPC, cache
from test_kv_step_host import append, attend, scales


def test_scales_lead_to_no_element_2_to_the_30():
    c = cache(dtype=4, heads=4, table=1 << 23, page=32, pages=3, tokens=64)
    last = lambda s: 2 * s[0] + s[1] + 3 * s[2]  # noqa: E731
    near, far = ((2 ** 30 - 8) // 2, 4, 1), ((2 ** 30 - 8) // 2, 5, 1)
    assert last(near) == 2 ** 30 - 1 and last(far) == 2 ** 30
    for name in ("ks", "vs"):
        assert attend(c, scales(**{name: near}), ws_bytes=0) == ENOSPC
        assert attend(c, scales(**{name: far}), ws_bytes=0) == EINVAL
        assert append(c, scales(**{name: far})) == EINVAL
