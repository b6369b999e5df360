"""The option that chooses the selective scan's form."""
import pytest

from linear_attention_recurrence_gb300 import gdn


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrence_gb300 import build

    build.build()
    return gdn.load_library()


def test_scan_form_option(lib):
    assert gdn.gdn_get_option("ssm_scan_form") == 0
    with gdn.options(ssm_scan_form=1):
        assert gdn.gdn_get_option(gdn.GDN_OPT_SSM_SCAN_FORM) == 1
    assert gdn.gdn_get_option("ssm_scan_form") == 0
    for value in (-1, 2):
        assert lib.gdn_set_option(gdn.GDN_OPT_SSM_SCAN_FORM, value) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.gdn_get_option("ssm_scan_form") == 0
