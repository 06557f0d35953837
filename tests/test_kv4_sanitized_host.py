"""The host checks of the rotary positions and of the cache in four bits with the C-ABI sources' host pass under
AddressSanitizer and UBSan (CPU only)."""
import os

import pytest


@pytest.mark.parametrize("checks", ["test_rotary_cpu.py", "test_kv4_abi_cpu.py"])
def test_host_checks_under_sanitizers(tmp_path, monkeypatch, checks):
    host = pytest.importorskip("test_attention_sanitized_host")
    monkeypatch.setattr(host, "CHECKS", os.path.join(os.path.dirname(os.path.abspath(__file__)), checks))
    host.test_host_checks_under_sanitizers(tmp_path)
