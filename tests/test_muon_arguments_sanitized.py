"""The Muon argument tests against a host-only build of the library with
AddressSanitizer and UndefinedBehaviorSanitizer (CPU, no GPU)."""
from test_muon_sanitizers import _preamble, _run, library, pytestmark  # noqa: F401


def test_argument_checks_under_sanitizers(library):  # noqa: F811
    out = _run(_preamble(library) + "import pytest; sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', "
                                    "'tests/test_muon_arguments.py']))")
    assert " passed" in out
