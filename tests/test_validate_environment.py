"""CPU tests of the switch for the value checks: os.environ as it is at the call."""
import os
from unittest import mock

import pytest

import structured_state_space_dplr_amd as s4


class Other:
    """A mapping of another kind, with an attribute of the interpreter's one."""
    _data = {b"S4DPLR_VALIDATE": b"1"}

    def get(self, name, default=None):
        return default


@pytest.mark.parametrize("env,want", [({"S4DPLR_VALIDATE": "1"}, True), ({"S4DPLR_VALIDATE": "0"}, False), ({}, False),
                                      (Other(), False)])
@pytest.mark.parametrize("own", ["0", "1"])
def test_environment_that_was_replaced(monkeypatch, env, want, own):
    """A mapping in os.environ's place is what counts."""
    monkeypatch.setenv("S4DPLR_VALIDATE", own)
    assert s4.validation_enabled() == (own == "1")
    with mock.patch.object(os, "environ", env):
        got = s4.validation_enabled()
    assert got == want
