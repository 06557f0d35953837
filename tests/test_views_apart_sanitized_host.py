"""The host checks of views apart of one buffer and of far frequencies with the C-ABI sources' host pass under
AddressSanitizer and UBSan (CPU only)."""
import os

import pytest


@pytest.mark.parametrize("checks", ["test_views_apart_cpu.py", "test_rotary_far_cpu.py"])
def test_host_checks_under_sanitizers(tmp_path, monkeypatch, checks):
    host = pytest.importorskip("test_attention_sanitized_host")
    monkeypatch.setattr(host, "CHECKS", os.path.join(os.path.dirname(os.path.abspath(__file__)), checks))
    host.test_host_checks_under_sanitizers(tmp_path)
