"""What the device sources may not hold."""
import glob
import os
import re

import trellis_quantized_moe_sort_gb300 as tq

CSRC = os.path.join(os.path.dirname(tq.__file__), "csrc")


def test_no_copy_to_several_ctas():
    """A bulk copy to several CTAs at once may only read the memory of its own GPU, and the
    addresses behind a tensor map are the caller's: the library has no such copy."""
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")))
    assert len(sources) > 10
    copies = 0
    for path in sources:
        with open(path) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())   # instructions written over several literals
        for line in text.splitlines():
            if "cp.async.bulk" in line:
                copies += 1
                assert "multicast" not in line, (os.path.basename(path), line)
    assert copies > 5
