"""The paged cache's and the attentions' validation under the host sanitizers (CPU; see test_host_sanitizers.py)."""

import pytest

import test_host_sanitizers as base


@pytest.mark.parametrize("kind", sorted(base.SANITIZERS))
def test_cache_entry_points_under_sanitizer(kind, tmp_path, monkeypatch):
    monkeypatch.setattr(base, "TESTS", ["tests/test_cache_abi.py"])
    base.test_host_code_under_sanitizer(kind, tmp_path)
