"""When the Python binding is built anew."""
import os

import torch

from lightning_indexer_b200 import build


def test_binding_follows_torch(monkeypatch):
    """A binding built against another torch is stale, although no source is newer."""
    monkeypatch.setattr(os.path, "getmtime", lambda f: 0.0)
    assert not build.needs_binding()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert build.needs_binding()
