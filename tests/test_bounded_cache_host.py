"""The calls after the verify attention, refused for how their buffers lie: no GPU needed, nothing is launched."""
import numpy as np
import pytest

from test_step_host import SELECT, pkv  # noqa: F401


def refused(pkv, call, values, word):  # noqa: F811
    status = getattr(pkv.lib, call)(*values.values())
    assert status == pkv.PKV_ERR_INVALID_ARG and word in pkv.lib.pkv_last_error(), (status, pkv.lib.pkv_last_error())


@pytest.mark.parametrize("change", [
    dict(nl=0x1000),                          # the lengths updated in place
    dict(nl=0x1004), dict(nl=0x0ffc),         # a part of them
    dict(keep=0x1000), dict(keep=0x1004), dict(keep=0x1000 - 4 * 2 * 4 * 8 + 4),
    dict(nl=0x2000 + 4 * 2 * 4 * 8 - 4), dict(nl=0x2000 - 4),
])
def test_select_refuses_outputs_over_its_lengths(pkv, change):  # noqa: F811
    """Every CTA of a request reads its length while one of them writes the new one."""
    base = {**SELECT, "s": 0x100000, "R": 2, "sl": 0x1000, "keep": 0x2000, "nl": 0x3000}
    refused(pkv, "pkv_kv_evict_select", {**base, **change}, b"overlap")
