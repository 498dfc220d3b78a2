"""The page lists of an attention plan: never read past the bounds that the
caller gave."""
import pytest

from test_host_cpu import SANITIZE, _native_check


@pytest.mark.parametrize("flags", [[], SANITIZE], ids=["plain", "asan_ubsan"])
def test_bounds_are_checked_before_the_lists_are_read(tmp_path, flags):
    _native_check(tmp_path, "attend_lists_check", "attend_plan.cpp", flags)
