"""The records that carry the fixed-state mixers' arguments to the library (no GPU)."""
import ctypes
import struct

import pytest

from tests.test_capi_host import cla

__all__ = ["cla"]


def test_a_library_with_other_records_is_refused(cla, monkeypatch):
    """One field more or less in any of them is noticed when the library is loaded, before
    a call could read behind a record."""
    lib = ctypes.CDLL(cla.LIB_PATH)
    cla._declare(lib)
    for at, record in enumerate(cla._RECORDS):
        for other in (record.format + "i", record.format + "P", "@8P"):
            changed = list(cla._RECORDS)
            changed[at] = struct.Struct(other)
            monkeypatch.setattr(cla, "_RECORDS", tuple(changed))
            with pytest.raises(RuntimeError, match="build it again"):
                cla._declare(lib)
