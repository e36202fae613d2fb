"""A page choice that no call accepts is refused where it is made, or where the step is
built that has it."""

import dataclasses

import numpy as np
import pytest

from speculative_decoding_verification_padding_gb300 import build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep, PageChoice


@pytest.mark.parametrize("values", [(0,), (-3,), (1025,), (4,), (5, 2, 4), (5, -1, 4), (5, 1, -1)])
def test_values_that_are_refused(values):
    with pytest.raises(ValueError):
        PageChoice(*values)


@pytest.mark.parametrize("values", [(5,), (1, 0, 0), (1, 1, 0), (1024, 1000, 24), (8, 4, 4)])
def test_values_that_are_taken(values):
    c = PageChoice(*values)
    assert c.n_keep == values[0]


@pytest.mark.gpu
def test_a_table_that_is_too_wide():
    build.build()
    w = wl.make_workload(wl.config("batch64"), n_req=1, ctx_scale=0.01, vocab=512)
    room = 49152 - w.block_tables.shape[1]
    wide = [np.pad(w.block_tables, ((0, 0), (0, n)), constant_values=-1) for n in (room, room + 1)]
    s = DeviceStep(dataclasses.replace(w, block_tables=wide[0]), mode="onepass", choice=PageChoice(5, 1, 1))
    s.run()
    assert s.results()["dev_status"] == 0
    with pytest.raises(ValueError):
        DeviceStep(dataclasses.replace(w, block_tables=wide[1]), mode="onepass", choice=PageChoice(5, 1, 1))
