"""kvc_rope_init at the ends of what doubles hold: what a float or a turn cannot hold is refused."""
import pytest

from tests.test_prompt_ops import lib  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(magnitude=1e39), dict(magnitude=1e-39), dict(magnitude=1e300), dict(magnitude=1e-300),
    dict(scaling="ntk", factor=1e-320), dict(scaling="ntk", factor=1e308, base=1e300),
    dict(scaling="linear", factor=1e-320), dict(scaling="linear", factor=1e-20),
    dict(scaling="bands", factor=1e-310, original=8192.0), dict(scaling="bands", factor=1e-20, original=8192.0),
    dict(scaling="ntk", factor=1e-30)])
def test_what_cannot_be_held_is_refused(lib, kw):  # noqa: F811
    """Magnitudes that are infinite or below the normal numbers as a float; frequencies that are not
    finite, or so fast (2^32 turns a token) that their part of a turn is lost."""
    import eviction_gb300 as kvc
    with pytest.raises(kvc.KvcError, match="KVC_ERR_ARG"):
        kvc.Rope(64, **kw)


@pytest.mark.parametrize("kw", [dict(magnitude=3e38), dict(magnitude=2e-38), dict(scaling="linear", factor=1e-9),
                                dict(scaling="ntk", factor=1e-2), dict(base=1e300), dict(scaling="linear", factor=1e300),
                                dict(scaling="bands", factor=1e300, original=8192.0)])
def test_what_can_be_held_is_taken(lib, kw):  # noqa: F811
    import eviction_gb300 as kvc
    r = kvc.Rope(64, **kw)
    assert any(r._c.turn) or kw.get("factor") == 1e300 and kw["scaling"] == "linear"
