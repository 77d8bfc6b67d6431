"""Every status that a call stores or returns has a name, whichever call is asked for it."""
import pytest

import rmsnorm_fp4_quant_gb300 as fq
from rmsnorm_fp4_quant_gb300 import build as fbuild


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    return fq.lib()


def test_no_pages_has_a_name():
    L = fq.lib()
    assert b"page" in L.fp4_status_string(fq.FP4_ERR_NO_PAGES)
    for status in range(8):
        assert L.fp4_status_string(status) == L.fp4_kv_status_string(status)
