"""The host-side validation of adapters and checkpoints under AddressSanitizer and
UndefinedBehaviorSanitizer, as that of the other operators: lh_api.hip rebuilt
with host-only sanitizers and the boundary tests run against it."""
import pytest

import test_host_sanitize_operators as operators
from test_host_sanitize import HIPCC, _asan_runtime

import os


@pytest.mark.skipif(not os.path.exists(HIPCC) or _asan_runtime() is None, reason="hipcc or its ASan runtime missing")
def test_adapters_validation_is_clean_under_sanitizers(monkeypatch):
    monkeypatch.setattr(operators, "TESTS", ["test_boundary_lora.py"])
    operators.test_operators_validation_is_clean_under_sanitizers()
