"""The marshalling extension: which file it is, and who needs it. No GPU."""
import importlib.machinery
import os

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD


def test_extension_carries_the_interpreters_tag():
    """A copy built for another Python has another name and is not loaded."""
    BLD.build()
    assert B.MARSHAL_PATH == BLD.MARSHAL and os.path.exists(BLD.MARSHAL)
    name = os.path.basename(BLD.MARSHAL)
    assert name.startswith("_marshal.cpython-") and name.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
