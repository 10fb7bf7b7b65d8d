import builtins
import os
import sys
import zlib

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
# A copy of oracle/ with a planted mistake (tests/test_oracle_mutants.py) is
# imported in place of oracle/ when its directory is named here.
if os.environ.get("HG_ORACLE_DIR"):
    sys.path.insert(0, os.environ["HG_ORACLE_DIR"])


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


@pytest.fixture(scope="session")
def oracle():
    from oracle import hashgrid_oracle
    return hashgrid_oracle


def repeatable_hash(key):
    """hash(key); of a key with texts in it, whose hash Python salts anew in each process, one that stays."""
    texts = any(isinstance(k, str) for k in (key if isinstance(key, tuple) else (key,)))
    return zlib.crc32(repr(key).encode()) if texts else builtins.hash(key)


@pytest.fixture(autouse=True)
def _seeds_that_stay(request, monkeypatch):
    """A test that seeds its inputs with hash() of its parameters has the same inputs in each run."""
    if not hasattr(request.module, "hash"):
        monkeypatch.setattr(request.module, "hash", repeatable_hash, raising=False)
