"""The host checks of views apart of one buffer with the C-ABI sources' host pass under AddressSanitizer and UBSan (CPU
only)."""
import os

import pytest


def test_host_checks_under_sanitizers(tmp_path, monkeypatch):
    host = pytest.importorskip("test_attention_sanitized_host")
    monkeypatch.setattr(host, "CHECKS", os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_views_apart_cpu.py"))
    host.test_host_checks_under_sanitizers(tmp_path)
