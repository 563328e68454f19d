"""The range-checked build under the norm's, rotary's and the 4-bit cache's tests: their kernels check the cache rows
that tables and ids name and the places of shared memory that positions and units take (the norm's places are its launch's
alone: it has none to check).  Every test passes there, and no check has failed when they are through."""
import os

import pytest

from test_gpu_checked import HERE, _child, checked_lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

CODE = """
import sys
import pytest
rc = pytest.main(["-x", "-q", "-p", "no:cacheprovider", *sys.argv[1:]])
from sparse_attention_gemm_gb300 import ops
status = ops.device_status(clear=True)
assert rc == 0 and status == 0, (rc, hex(status))
"""


@pytest.mark.parametrize("names,skip", [(("test_gpu_rows.py",), "many_rows"),
                                        (("test_gpu_kv4.py", "test_gpu_attention_edges.py"), "32_bits or threads or 8_bit_cache")])
def test_rows_and_4_bit_cache_on_the_checked_build(checked_lib, names, skip):  # noqa: F811
    r = _child(["-c", CODE, *(os.path.join(HERE, n) for n in names), "-k", f"not ({skip})"], checked_lib)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-2000:])
