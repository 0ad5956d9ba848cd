"""The sanitizer tests are there to be run: a module that takes the driver of
another by importorskip would show a broken import as a skip."""

import importlib
import os

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name", ["test_host_sanitize", "test_packed_sanitize"])
def test_sanitizer_modules_import(name):
    module = importlib.import_module(f"tests.{name}")
    assert callable(getattr(module, "driver")) and os.path.dirname(module.__file__) == HERE
